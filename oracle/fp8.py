"""Oracle: e4m3 codes with a scale per block of 128, and the layer over them (test
infrastructure only).

e4m3 has 1 sign, 4 exponent (bias 7) and 3 fraction bits, no infinities, NaN as exponent and
fraction all ones; its finite magnitudes end at 448 and its subnormal step is 2^-9.

A block's scale and codes: a = max(max|x|, 2^-100), s = fl32(a/448), and each code is the e4m3
value nearest to x·448/a, halves to even (the fp64 quotient of fp32 values is never rounded onto
a tie or off one: it is one or at least 2^-30 of itself away). A block that holds a
NaN or an infinity has s = NaN and NaN codes. Blocks are 1 x 128 (activations) or 128 x 128
(weights), cut off at the matrix's edges.

The layer: Y[t][o] = Σ_c (code·s)(X)[t][c] · (code·s)(W)[o][c] + R[t][o], in fp64.
"""

import numpy as np


def e4m3_round(v):
    """The e4m3 value nearest to each v (halves to even, magnitudes end at 448), in fp64."""
    v = np.asarray(v, np.float64)
    _, e = np.frexp(np.where(v == 0.0, 1.0, v))             # |v| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def quantize(x, rows):
    """(values of the codes fp64 [n, d], scales float32 [ceil(n/rows), ceil(d/128)])."""
    x = np.asarray(x, np.float64)
    n, d = x.shape
    nr, nb = -(-n // rows), -(-d // 128)
    codes = np.empty((n, d))
    scales = np.empty((nr, nb), np.float32)
    for i in range(nr):
        for b in range(nb):
            at = np.s_[i * rows:(i + 1) * rows, b * 128:(b + 1) * 128]
            blk = x[at]
            if not np.all(np.isfinite(blk)):
                codes[at], scales[i, b] = np.nan, np.nan
                continue
            a = np.float32(max(np.max(np.abs(blk)), 2.0 ** -100))
            scales[i, b] = a / np.float32(448.0)
            codes[at] = e4m3_round(blk * 448.0 / np.float64(a))
    return codes, scales


def quantize_act(x):
    """As the layer stores it: scales [ceil(d/128), n]."""
    codes, scales = quantize(x, 1)
    return codes, np.ascontiguousarray(scales.T)


def quantize_weight(w):
    return quantize(w, 128)


def dequant(codes, scales, rows):
    """code · scale in fp64, scales [row blocks, column blocks]."""
    n, d = codes.shape
    s = np.asarray(scales, np.float64)[np.arange(n) // rows][:, np.arange(d) // 128]
    return np.asarray(codes, np.float64) * s


def linear(x_codes, x_scales, w_codes, w_scales, R=None):
    """(Y, Σ_c |x̂·ŵ|) in fp64; the second is what the error of a summation scales with."""
    X = dequant(x_codes, np.asarray(x_scales).T, 1)
    W = dequant(w_codes, w_scales, 128)
    Y = X @ W.T
    return (Y if R is None else Y + np.asarray(R, np.float64)), np.abs(X) @ np.abs(W).T
