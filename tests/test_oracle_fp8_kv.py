"""Pins of the oracle's e4m3 blocks and of its quantised cache against something other than
themselves: torch's e4m3 conversion, brute force over the code values, the quantizer's bound, and
the RTN oracle. And the host-side refusals of the library's calls, which launch nothing."""

import os

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle import kv_cache as okv
from oracle import rtn as ortn

E4M3_VALUES = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
FINITE = np.unique(E4M3_VALUES[np.isfinite(E4M3_VALUES)])


def test_e4m3_round_is_the_nearest_value_with_even_ties():
    rng = np.random.default_rng(0)
    v = np.concatenate([rng.normal(size=2000) * 10.0 ** rng.uniform(-4, 2, 2000), FINITE,
                        (FINITE[1:] + FINITE[:-1]) / 2, [0.0, -0.0, 448.0, 1e-9]])
    v = v[np.abs(v) <= 448.0]
    got = ofp8.e4m3_round(v)
    assert np.all(np.isin(got, FINITE))
    best = np.min(np.abs(v[:, None] - FINITE[None, :]), axis=1)
    assert np.array_equal(np.abs(got - v), best)
    ref = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    same32 = v.astype(np.float32).astype(np.float64) == v
    assert np.array_equal(got[same32], ref[same32])           # ties to even among them


@pytest.mark.parametrize("rows", [1, 128])
def test_block_quantizer_is_within_half_a_step(rows):
    """|x - code·s| <= half an e4m3 step of the scaled value (2^-4 relative, 2^-10 in the subnormal
    range) plus the three fp32 roundings of s, r and x·r (3·2^-24 relative)."""
    rng = np.random.default_rng(rows)
    x = (rng.normal(size=(130, 272)) * np.exp(rng.normal(size=272))).astype(np.float16)
    codes, scales = ofp8.quantize(x, rows)
    assert scales.shape == (-(-130 // rows), 3) and np.all(np.isin(codes, FINITE))
    s = np.repeat(np.repeat(scales.astype(np.float64), rows, 0)[:130], 128, 1)[:, :272]
    xd = x.astype(np.float64)
    tol = np.maximum(2.0 ** -4 * np.abs(xd), 2.0 ** -10 * s) + 3 * 2.0 ** -24 * np.abs(xd)
    assert np.all(np.abs(codes * s - xd) <= tol)
    assert np.max(np.abs(codes)) == 448.0


def test_block_quantizer_edge_blocks():
    x = np.zeros((3, 256), np.float32)
    x[0, 128:] = 1e-38
    x[1, 5] = np.inf
    x[2, 200] = np.nan
    codes, scales = ofp8.quantize(x, 1)
    floor = np.float32(2.0 ** -100) / np.float32(448.0)
    assert np.all(codes[0] == 0) and np.all(scales[0] == floor)
    assert np.all(np.isnan(codes[1, :128])) and np.isnan(scales[1, 0]) and scales[1, 1] == floor
    assert scales[2, 0] == floor and np.all(np.isnan(codes[2, 128:])) and np.isnan(scales[2, 1])


def test_linear_against_a_loop():
    rng = np.random.default_rng(3)
    xc, xs = ofp8.quantize_act(rng.normal(size=(3, 144)))
    wc, ws = ofp8.quantize_weight(rng.normal(size=(130, 144)))
    R = rng.normal(size=(3, 130))
    Y, mag = ofp8.linear(xc, xs, wc, ws, R)
    for t, o in ((0, 0), (2, 129), (1, 77)):
        terms = [xc[t, c] * float(xs[c // 128, t]) * wc[o, c] * float(ws[o // 128, c // 128])
                 for c in range(144)]
        assert abs(Y[t, o] - (sum(terms) + R[t, o])) < 1e-12
        assert abs(mag[t, o] - sum(abs(v) for v in terms)) < 1e-12


@pytest.mark.parametrize("bits,g", [(4, 16), (8, 32), (4, 64), (8, 128)])
def test_cache_quantizer_is_the_rtn_quantizer(bits, g):
    rng = np.random.default_rng(bits * g)
    x = (rng.normal(size=(5, 2, 128)) * 3.0).astype(np.float16)
    q, s, z = okv.quantize(x, bits, g)
    rc, rs, rz = ortn.rtn_minmax(x.reshape(10, 128).astype(np.float64), bits, g)
    assert np.array_equal(q.reshape(10, 128), rc)
    assert np.array_equal(s.reshape(10, -1), rs) and np.array_equal(z.reshape(10, -1), rz)
    err = np.abs(np.repeat(s, g, -1) * (q - np.repeat(z, g, -1)) - x.astype(np.float64))
    assert np.all(err <= np.repeat(s, g, -1) / 2)


def test_cache_write_and_read_round_trip():
    rng = np.random.default_rng(9)
    H, D, g, page, n_pages = 2, 32, 16, 3, 7
    codes = np.zeros((2, n_pages, page, H, D // 2), np.uint8)
    scales = np.zeros((2, n_pages, page, H, D // g), np.float16)
    zeros = np.zeros_like(scales)
    K, V = rng.normal(size=(2, 9, H, D)).astype(np.float16)
    table = np.array([[4, 1], [0, -1], [6, 2]])
    lens = [5, 0, 4]
    slots = [table[b][p // page] * page + p % page for b in range(3) for p in range(lens[b])]
    okv.write(codes, scales, zeros, K, V, slots, 4)
    k, v = okv.read(codes, scales, zeros, table, np.cumsum([0] + lens), 4)
    for got, x in ((k, K), (v, V)):
        q, s, z = okv.quantize(x, 4, g)
        assert np.array_equal(got, np.repeat(s, g, -1) * (q - np.repeat(z, g, -1)))
    assert not codes[:, 3].any() and not codes[:, 5].any()         # pages of nobody
    bad = np.full((1, 1, 16), np.nan, np.float16)
    q, s, z = okv.quantize(bad, 8, 16)
    assert not q.any() and np.isnan(s).all() and not z.any()


# ------------------------------------------------------------------------------------------
# refusals (host side, nothing is launched)
# ------------------------------------------------------------------------------------------
@pytest.fixture(scope="module")
def L():
    from post_weight_quantization_24_b200 import build, gptq
    build.build()
    return gptq.lib()


ERR_ARG = -1
P = 4096     # stands for a device pointer; every call below fails a check before using it


def test_fp8_refusals(L):
    def act(X=P, dt=0, n=4, d=128, c=P, s=P):
        return L.fp8_quantize_act(X, dt, n, d, c, s, None)

    def weight(W=P, dt=0, o=4, d=128, c=P, s=P):
        return L.fp8_quantize_weight(W, dt, o, d, c, s, None)

    def linear(X=P, sx=P, n=4, d=128, W=P, sw=P, o=4, R=None, Y=P, dt=0, st=None):
        return L.fp8_linear(X, sx, n, d, W, sw, o, R, Y, dt, st, None)

    for kw in (dict(X=None), dict(dt=3), dict(dt=-1), dict(n=-1), dict(n=1 << 31), dict(d=0),
               dict(d=24), dict(d=65552), dict(c=None), dict(s=None), dict(X=P + 8), dict(c=P + 4),
               dict(s=P + 2)):
        assert act(**kw) == ERR_ARG, kw
    assert act(n=0, X=None, c=None, s=None) == 0                   # nothing to do
    for kw in (dict(W=None), dict(dt=3), dict(o=0), dict(d=8), dict(d=40), dict(d=65552),
               dict(c=None), dict(s=None), dict(W=P + 2), dict(c=P + 8), dict(s=P + 1)):
        assert weight(**kw) == ERR_ARG, kw
    for kw in (dict(X=None), dict(sx=None), dict(W=None), dict(sw=None), dict(Y=None), dict(n=-1),
               dict(n=1 << 31), dict(d=8), dict(d=100), dict(d=65552), dict(o=0), dict(dt=3),
               dict(X=P + 8), dict(W=P + 8), dict(Y=P + 8), dict(R=P + 8), dict(sx=P + 2),
               dict(sw=P + 2), dict(st=P + 2)):
        assert linear(**kw) == ERR_ARG, kw
    assert linear(n=0, X=None, sx=None, Y=None) == 0


def test_kv_cache_refusals(L):
    def write(K=P, V=P, dt=0, n=4, ks=256, vs=256, H=2, D=128, slots=P, ns=64, bits=8, g=64, c=P,
              s=P, z=P, st=None):
        return L.kv_cache_write(K, V, dt, n, ks, vs, H, D, slots, ns, bits, g, c, s, z, st, None)

    def read(c=P, s=P, z=P, npg=4, ps=16, H=2, D=128, bits=8, g=64, tab=P, ns=2, mp=3, cu=P,
             total=7, K=P, V=P, dt=0, st=None):
        return L.kv_cache_read(c, s, z, npg, ps, H, D, bits, g, tab, ns, mp, cu, total, K, V, dt,
                               st, None)

    shared = (dict(dt=3), dict(H=0), dict(D=8, g=16), dict(D=120), dict(H=1024, D=128),
              dict(bits=3), dict(bits=16), dict(g=8), dict(g=48, D=96), dict(g=512, D=512),
              dict(g=0), dict(c=None), dict(s=None), dict(z=None), dict(c=P + 8), dict(s=P + 1),
              dict(z=P + 1), dict(K=None), dict(V=None), dict(K=P + 8), dict(V=P + 8),
              dict(st=P + 2))
    for kw in shared + (dict(n=-1), dict(n=1 << 31), dict(ks=-8), dict(vs=12), dict(ks=1 << 32),
                        dict(slots=None), dict(slots=P + 4), dict(ns=0), dict(dt=1, ks=258)):
        assert write(**kw) == ERR_ARG, kw
    for kw in shared + (dict(npg=0), dict(npg=1 << 31), dict(ps=0), dict(ns=-1), dict(mp=-1),
                        dict(total=-1), dict(total=1 << 31), dict(tab=None), dict(cu=None),
                        dict(tab=P + 2), dict(cu=P + 2)):
        assert read(**kw) == ERR_ARG, kw
    assert write(n=0, K=None, V=None, slots=None) == 0
    assert read(total=0, K=None, V=None) == 0
    assert read(ns=0, tab=None, cu=None) == 0


def test_host_tensors_are_refused():
    from post_weight_quantization_24_b200 import gptq
    x = torch.zeros(4, 128, dtype=torch.float16)
    x8 = x.to(torch.float8_e4m3fn)
    s = torch.ones(1, 4)
    cache = gptq.kv_cache_alloc(2, 4, 1, 64, device="cpu")
    for call in (lambda: gptq.fp8_quantize_act(x), lambda: gptq.fp8_quantize_weight(x),
                 lambda: gptq.fp8_linear(x8, s, x8, s[:, :1]),
                 lambda: gptq.kv_cache_write(x.view(4, 1, 128), x.view(4, 1, 128),
                                             torch.zeros(4, dtype=torch.int64), *cache),
                 lambda: gptq.kv_cache_read(*cache, torch.zeros(1, 1, dtype=torch.int32),
                                            torch.zeros(2, dtype=torch.int32), 0)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_header_names_the_calls(L):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "gptq.h")).read()
    for name in ("fp8_quantize_act", "fp8_quantize_weight", "fp8_linear", "kv_cache_write",
                 "kv_cache_read"):
        assert f"gptq_status {name}(" in text and hasattr(L, name)
