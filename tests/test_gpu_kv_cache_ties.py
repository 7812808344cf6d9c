"""Exact ties of the cache's codes and their neighbours.

Groups whose range is exactly (2^bits - 1)·2^k get the scale 2^k, and values (j + 1/2)·2^k lie
halfway between two codes: rint takes the even one before the zero point is added. Every group
holds both ends of its range and, between them, ties (and with ``by`` = 1 or -1 the values next to
them), for even and odd j, in both signs. Codes, scales and zeros are compared bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import kv_cache as okv

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _np(t):
    return t.detach().cpu().double().numpy()


def _groups(n_groups, g, bits, k, dtype, by):
    """([n_groups, g] values, how many of them are ties)."""
    maxq = 2 ** bits - 1
    rng = np.random.default_rng(1000 * bits + g)
    lows = [0, -maxq, -(maxq // 2), -(maxq // 2 + 1), -1, -3]
    out = torch.empty(n_groups, g, dtype=dtype)
    ties = 0
    for i in range(n_groups):
        lo = lows[i % len(lows)]
        hi = lo + maxq
        half = np.arange(lo, hi) + 0.5
        t = torch.from_numpy(half * 2.0 ** k).to(dtype)
        t = t[t.double() == torch.from_numpy(half * 2.0 ** k)]         # those that the type has
        t = t[torch.from_numpy(rng.permutation(np.resize(rng.permutation(len(t)), g - 2)))]
        if by:
            t = (t.view(torch.int32 if dtype == F32 else torch.int16) + by).view(dtype)
        out[i, 0], out[i, 1] = lo * 2.0 ** k, hi * 2.0 ** k
        out[i, 2:] = t
        frac = _np(t) / 2.0 ** k
        ties += int(np.sum(np.abs(frac - np.floor(frac)) == 0.5))
    return out, ties


@pytest.mark.parametrize("dtype,powers", [(F16, (-13, 0, 3)), (BF16, (-24, -13, 0, 7)),
                                          (F32, (-24, -13, 0, 7))])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("H,D,g", [(1, 48, 16), (3, 64, 32), (1, 256, 256), (4, 128, 64),
                                   (8, 128, 128), (8, 128, 16), (4, 256, 32)])
def test_codes_of_ties_and_their_neighbours(cuda_lib, H, D, g, bits, dtype, powers):
    n, page = 12, 4
    for k in powers:
        for by in (0, 1, -1):
            x, ties = _groups(2 * n * H * D // g, g, bits, k, dtype, by)
            if by == 0:
                assert ties == x.shape[0] * (g - 2)
            K, V = x.view(2, n, H, D)
            q, s, z = okv.quantize(_np(K), bits, g)
            assert np.all(s == 2.0 ** k)
            dev = cuda_lib.kv_cache_alloc(n // page, page, H, D, bits, g)
            host = [t.cpu().numpy() for t in dev]
            cuda_lib.kv_cache_write(K.cuda(), V.cuda(), torch.arange(n, device="cuda"), *dev, bits=bits)
            okv.write(*host, _np(K), _np(V), list(range(n)), bits)
            for d, h in zip(dev, host):
                assert np.array_equal(d.cpu().numpy(), h), (k, by)
