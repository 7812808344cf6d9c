"""The e4m3 block quantizers and the layer over them against the fp64 oracle.

Codes and scales are compared bit for bit: the definition is three fp32 operations and one e4m3
rounding, all correctly rounded on both sides.

Tolerance of the layer, from the arithmetic. Products of e4m3 codes are exact. The tensor cores
add 32 of them to the accumulator per instruction; a sum that is aligned to its largest term and
cut to 24 bits loses less than 2^-23 of the largest term for each of its 33 terms, and 4
instructions make a block, so a block's sum is off by less than 4·33·2^-23 of its Σ|x·w|. (The
legacy instructions of the short form take two times 16 terms: fewer.) The factor sx·sw, the
fused multiply-adds over nb blocks, the joining of up to 16 partial sums and the residual's
addition are off by 2^-24 each, relative to Σ|x̂·ŵ| (+ |R|). One rounding to Y's type is off by
half a step.
"""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _values(n, d, seed, dtype=F16, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, d, generator=g) * torch.exp(spread * torch.randn(d, generator=g))
    return x.to(dtype)


def _np(t):
    return t.detach().cpu().double().numpy()


def _same(got, ref):
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.array_equal(got[ok], ref[ok]), int(np.sum(got[ok] != ref[ok]))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("n,d", [(1, 16), (1, 4096), (4, 128), (33, 144), (130, 1040), (257, 112)])
def test_quantizers_match_the_oracle(cuda_lib, n, d, dtype):
    x = _values(n, d, seed=n + d, dtype=dtype)
    codes, scales = cuda_lib.fp8_quantize_act(x.cuda())
    rc, rs = ofp8.quantize_act(_np(x))
    _same(_np(codes), rc)
    _same(_np(scales), rs.astype(np.float64))
    codes, scales = cuda_lib.fp8_quantize_weight(x.cuda())
    rc, rs = ofp8.quantize_weight(_np(x))
    _same(_np(codes), rc)
    _same(_np(scales), rs.astype(np.float64))


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_quantizers_on_edge_blocks(cuda_lib, dtype):
    """Zero blocks, the type's smallest and largest values, signed zeros, NaN and infinities: each
    stays in its own block."""
    fi = torch.finfo(dtype)
    x = _values(140, 400, seed=5, dtype=dtype)
    x[0] = 0.0
    x[1, :128] = -0.0
    x[2] = fi.smallest_normal
    x[3] = -fi.smallest_normal * fi.eps
    x[4, 3], x[4, 7] = fi.max, -fi.max
    x[5, 130] = float("nan")
    x[6, 399] = float("inf")
    x[7, 0] = -float("inf")
    x[135, 260] = float("nan")
    for name, rows in (("fp8_quantize_act", 1), ("fp8_quantize_weight", 128)):
        codes, scales = getattr(cuda_lib, name)(x.cuda())
        rc, rs = ofp8.quantize(_np(x), rows)
        _same(_np(codes), rc)
        _same(_np(scales.t() if rows == 1 else scales), rs.astype(np.float64))


def test_quantizers_write_only_their_outputs(cuda_lib):
    """Given outputs inside larger buffers, on a stream of its own: nothing around them changes."""
    n, d = 37, 272
    x = _values(n, d, seed=2).cuda()
    buf = torch.full((n + 2, d), 0x55, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((5, n), -7.0, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        cuda_lib.fp8_quantize_act(x, out=(buf[1:-1].view(E4M3), sbuf[1:4]))
    st.synchronize()
    rc, rs = ofp8.quantize_act(_np(x))
    _same(_np(buf[1:-1].view(E4M3)), rc)
    _same(_np(sbuf[1:4]), rs.astype(np.float64))
    assert bool((buf[0] == 0x55).all()) and bool((buf[-1] == 0x55).all())
    assert bool((sbuf[0] == -7).all()) and bool((sbuf[4] == -7).all())


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("n,d", [(9, 1040), (3, 272), (1, 16)])
def test_quantize_rows_at_any_16_bytes(cuda_lib, n, d, dtype):
    """Inputs that start 16 bytes behind a 32-byte boundary get the same codes and scales."""
    x = _values(n, d, seed=n, dtype=dtype).cuda()
    skip = 16 // x.element_size()
    buf = torch.empty(n * d + 2 * skip, dtype=dtype, device="cuda")
    y = buf[skip:skip + n * d].view(n, d)
    y.copy_(x)
    assert y.data_ptr() % 32 == 16 and x.data_ptr() % 32 == 0
    for f in (cuda_lib.fp8_quantize_act, cuda_lib.fp8_quantize_weight):
        a, b = f(x), f(y)
        assert torch.equal(a[0].view(torch.uint8), b[0].view(torch.uint8))
        assert torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("n,d", [(8200, 4112), (1500, 5136), (5, 8208)])
def test_quantize_act_of_many_tokens_is_that_of_few(cuda_lib, n, d, dtype):
    """Every row's codes and scales are those of a call with a few rows, which are checked against
    the oracle above (a few here too)."""
    x = torch.randn(n, d, generator=torch.Generator(device="cuda").manual_seed(d), device="cuda")
    x = (x * torch.exp(torch.randn(d, generator=torch.Generator().manual_seed(n)).cuda())).to(dtype)
    x[n // 2, 17], x[n - 1, d - 1] = float("nan"), float("inf")
    codes, scales = cuda_lib.fp8_quantize_act(x)
    for r0 in (0, n // 2 - 2, n - 5):
        c, s = cuda_lib.fp8_quantize_act(x[r0:r0 + 5])
        assert torch.equal(c.view(torch.uint8), codes[r0:r0 + 5].view(torch.uint8))
        assert torch.equal(s.view(torch.int32), scales[:, r0:r0 + 5].contiguous().view(torch.int32))
        rc, rs = ofp8.quantize_act(_np(x[r0:r0 + 5]))
        _same(_np(c), rc)
        _same(_np(s), rs.astype(np.float64))
    step = max(1, n // 64)
    c, s = cuda_lib.fp8_quantize_act(x[::step].contiguous())
    assert torch.equal(c.view(torch.uint8), codes[::step].view(torch.uint8))
    assert torch.equal(s.view(torch.int32), scales[:, ::step].contiguous().view(torch.int32))


def _quantized(n, d_in, d_out, seed):
    xc, xs = ofp8.quantize_act(_np(_values(n, d_in, seed)))
    wc, ws = ofp8.quantize_weight(_np(_values(d_out, d_in, seed + 1, spread=0.3)))
    dev = [torch.from_numpy(a).float().to(E4M3).cuda() if i % 2 == 0 else torch.from_numpy(a).cuda()
           for i, a in enumerate((xc, xs, wc, ws))]
    return (xc, xs, wc, ws), dev


def _tolerance(mag, Y, R, d_in, dtype):
    nb = -(-d_in // 128)
    tol = (4 * 33 * 2.0 ** -23 + (nb + 18) * 2.0 ** -24) * mag
    if R is not None:
        tol = tol + 2.0 ** -24 * (np.abs(R) + mag)
    fi = torch.finfo(dtype)
    half_step = np.maximum(fi.eps / 2 * (np.abs(Y) + tol), fi.smallest_normal * fi.eps / 2)
    return tol + half_step


def _check_linear(lib, n, d_in, d_out, dtype, res, seed):
    host, dev = _quantized(n, d_in, d_out, seed)
    R = _values(n, d_out, seed + 2, dtype=dtype, spread=0.0) if res else None
    Y = lib.fp8_linear(*dev, R=None if R is None else R.cuda(), dtype=dtype)
    assert Y.dtype == dtype and Y.shape == (n, d_out)
    ref, mag = ofp8.linear(*host, R=None if R is None else _np(R))
    err = np.abs(_np(Y) - ref)
    tol = _tolerance(mag, ref, None if R is None else _np(R), d_in, dtype)
    assert np.all(err <= tol), (float(np.max(err / tol)), int(np.sum(~(err <= tol))))
    return dev, Y


@pytest.mark.parametrize("n", [1, 2, 5, 8, 9, 16, 17, 31, 33, 63, 64, 65, 100, 128, 129, 200, 257, 520])
@pytest.mark.parametrize("d_in,d_out,dtype,res", [(272, 264, F16, True), (1040, 100, BF16, False)])
def test_linear_over_token_counts(cuda_lib, n, d_in, d_out, dtype, res):
    _check_linear(cuda_lib, n, d_in, d_out, dtype, res, seed=n)


@pytest.mark.parametrize("n", [1, 3, 20, 70, 140, 300])
@pytest.mark.parametrize("d_in,d_out,dtype,res", [
    (16, 1, F16, False),          # the smallest layer
    (128, 8, F32, True),
    (144, 17, BF16, True),        # a block of 16 channels; odd rows of Y
    (2048, 131, F16, True),
    (4112, 516, F32, False),
    (640, 1000, BF16, False),
])
def test_linear_over_layer_shapes(cuda_lib, n, d_in, d_out, dtype, res):
    _check_linear(cuda_lib, n, d_in, d_out, dtype, res, seed=d_in + d_out)


@pytest.mark.parametrize("n,d_in,d_out", [(1, 11008, 4096), (48, 4096, 1032), (384, 8192, 640),
                                          (1500, 1024, 2056)])
def test_linear_on_large_layers(cuda_lib, n, d_in, d_out):
    _check_linear(cuda_lib, n, d_in, d_out, F16, True, seed=n)


@pytest.mark.parametrize("n,d_in,d_out,dtype,res", [
    (1030, 272, 2056, F16, True),         # ragged in tokens, channels and input channels
    (1030, 128, 2049, BF16, True),        # odd rows of Y
    (770, 400, 3300, F32, True),          # fp32 rows leave in two rounds
    (2600, 144, 4104, F16, False),        # several tiles per pair of SMs
    (2600, 144, 4104, BF16, True),
    (2600, 16, 4100, F32, True),
    (5000, 256, 1030, F16, False),
])
def test_linear_with_many_tiles(cuda_lib, n, d_in, d_out, dtype, res):
    """Calls with enough 256 x 256 tiles for pairs of SMs, the residual in place and not."""
    dev, Y = _check_linear(cuda_lib, n, d_in, d_out, dtype, res, seed=n)
    if res:
        R = _values(n, d_out, n + 2, dtype=dtype, spread=0.0).cuda()
        assert cuda_lib.fp8_linear(*dev, R=R, out=R) is R and torch.equal(R, Y)
    else:
        assert torch.equal(cuda_lib.fp8_linear(*dev, dtype=dtype), Y)


def test_offsets_past_32_bits(cuda_lib):
    """More than 2^31 elements of X, its codes and Y: the last rows are right."""
    n, d = 66000, 33024
    x = torch.empty(n, d, dtype=F16, device="cuda")
    tail = _values(3, d, seed=1)
    x[-3:] = tail.cuda()
    x[:-3] = 1.0
    codes, scales = cuda_lib.fp8_quantize_act(x)
    rc, rs = ofp8.quantize_act(_np(tail))
    _same(_np(codes[-3:]), rc)
    _same(_np(scales[:, -3:]), rs.astype(np.float64))
    wcodes, _ = cuda_lib.fp8_quantize_weight(x)
    assert bool((wcodes[:256].float() == 448).all())
    last = (n - 1) // 128 * 128
    rc, _ = ofp8.quantize_weight(_np(x[last:]))
    _same(_np(wcodes[last:]), rc)
    del x, codes, wcodes
    host, dev = _quantized(4, 16, d, seed=2)
    x8 = dev[0].repeat(n // 4, 1)
    sx = dev[1].repeat(1, n // 4)
    Y = cuda_lib.fp8_linear(x8, sx, dev[2], dev[3])
    assert Y.numel() > 1 << 31
    ref, mag = ofp8.linear(*host)
    assert np.all(np.abs(_np(Y[-4:]) - ref) <= _tolerance(mag, ref, None, 16, F16))
    assert torch.equal(Y[:4], Y[-4:])


@pytest.mark.parametrize("n", [1, 7, 12, 40, 90, 150, 600])
@pytest.mark.parametrize("d_in,d_out", [(272, 136), (1024, 1296)])
def test_linear_is_exact_on_small_integers(cuda_lib, n, d_in, d_out):
    """Codes in -3..3 and power-of-two scales: every sum is exact in fp32, so every bit of Y is
    determined, whatever the order of summation."""
    g = torch.Generator().manual_seed(n + d_in)
    nb, no = -(-d_in // 128), -(-d_out // 128)
    x8 = torch.randint(-3, 4, (n, d_in), generator=g).float().to(E4M3)
    w8 = torch.randint(-3, 4, (d_out, d_in), generator=g).float().to(E4M3)
    sx = 2.0 ** torch.randint(-2, 3, (nb, n), generator=g).float()
    sw = 2.0 ** torch.randint(-2, 3, (no, nb), generator=g).float()
    R = torch.randint(-8, 9, (n, d_out), generator=g).float()
    Y = cuda_lib.fp8_linear(x8.cuda(), sx.cuda(), w8.cuda(), sw.cuda(), R=R.cuda(), dtype=F32)
    ref, _ = ofp8.linear(_np(x8), sx.numpy(), _np(w8), sw.numpy(), R=_np(R))
    assert np.array_equal(_np(Y), ref)


@pytest.mark.parametrize("n", [1, 6, 37, 129, 300])
def test_linear_residual_in_place_and_rows_around_it(cuda_lib, n):
    d_in, d_out = 400, 200
    host, dev = _quantized(n, d_in, d_out, seed=n)
    buf = _values(n + 2, d_out, seed=8).cuda()
    before = buf.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = cuda_lib.fp8_linear(*dev, R=buf[1:-1], out=buf[1:-1], status=status)
    assert out.data_ptr() == buf[1:-1].data_ptr() and int(status) == 0
    ref, mag = ofp8.linear(*host, R=_np(before[1:-1]))
    tol = _tolerance(mag, ref, _np(before[1:-1]), d_in, F16)
    assert np.all(np.abs(_np(out) - ref) <= tol)
    assert torch.equal(buf[0], before[0]) and torch.equal(buf[-1], before[-1])


@pytest.mark.parametrize("n,d_out", [(3, 300), (20, 300), (150, 300), (2000, 2600)])
def test_linear_keeps_nan_to_its_token_and_channels(cuda_lib, n, d_out):
    """A token with a NaN block gives a NaN row; a weight block with NaN codes and scale gives NaN
    columns; nothing else changes."""
    host, dev = _quantized(n, 256, d_out, seed=1)
    clean = cuda_lib.fp8_linear(*dev)
    x8, sx, w8, sw = [t.clone() for t in dev]
    x8.view(torch.uint8)[1, 128:] = 0x7F
    sx[1, 1] = float("nan")
    w8.view(torch.uint8)[128:256, :128] = 0x7F
    sw[1, 0] = float("nan")
    Y = cuda_lib.fp8_linear(x8, sx, w8, sw)
    bad = torch.zeros(n, d_out, dtype=torch.bool, device="cuda")
    bad[1] = True
    bad[:, 128:256] = True
    assert torch.equal(torch.isnan(Y), bad)
    assert torch.equal(Y[~bad], clean[~bad])


@pytest.mark.parametrize("n,d_out", [(1, 520), (33, 520), (100, 520), (700, 520), (1300, 2304)])
def test_linear_repeats_its_bits_and_runs_from_a_graph(cuda_lib, n, d_out):
    """Equal inputs give equal bits; a captured call replays on new inputs, also while another
    call runs on another stream."""
    d_in = 2064
    _, dev = _quantized(n, d_in, d_out, seed=3)
    _, dev2 = _quantized(n, d_in, d_out, seed=30)
    want = [cuda_lib.fp8_linear(*d, dtype=F32) for d in (dev, dev2)]
    assert torch.equal(cuda_lib.fp8_linear(*dev, dtype=F32), want[0])
    ins = [t.clone() for t in dev]
    out = torch.empty(n, d_out, device="cuda")
    cuda_lib.fp8_linear(*ins, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cuda_lib.fp8_linear(*ins, out=out)
    for t, s in zip(ins, dev2):
        t.copy_(s)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        side = [cuda_lib.fp8_linear(*dev, dtype=F32) for _ in range(4)]
    for _ in range(4):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[1])
    assert all(torch.equal(s, want[0]) for s in side)


_CAPTURE_FIRST = """
import torch
from post_weight_quantization_24_b200 import gptq
x = torch.randn(200, 256, device='cuda').half()
cache = gptq.kv_cache_alloc(40, 16, 2, 64, 8, 64)
slots = torch.arange(200, device='cuda')
table = torch.arange(13, dtype=torch.int32, device='cuda').view(1, 13)
cu = torch.tensor([0, 200], dtype=torch.int32, device='cuda')
def run():
    w8, sw = gptq.fp8_quantize_weight(x)
    out = []
    for n in (1, 30, 60, 120, 200):
        out.append(gptq.fp8_linear(*gptq.fp8_quantize_act(x[:n]), w8, sw))
    big = x.repeat(8, 1)
    out.append(gptq.fp8_linear(*gptq.fp8_quantize_act(big), *gptq.fp8_quantize_weight(big)))
    kv = x[:, :128].unflatten(1, (2, 64))
    gptq.kv_cache_write(kv, kv, slots, *cache)
    return out + list(gptq.kv_cache_read(*cache, table, cu, 200))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    captured = run()
g.replay()
torch.cuda.synchronize()
again = run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(captured, again))
print('captured')
"""


def test_first_calls_may_be_captured(cuda_lib):
    """A process whose first calls are inside a capture: no warm-up is needed."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _CAPTURE_FIRST], cwd=root, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_empty_calls(cuda_lib):
    """No tokens: nothing is launched, and nothing is written."""
    x = torch.empty(0, 256, dtype=F16, device="cuda")
    codes, scales = cuda_lib.fp8_quantize_act(x)
    assert codes.shape == (0, 256) and scales.shape == (2, 0)
    _, dev = _quantized(2, 256, 40, seed=1)
    Y = cuda_lib.fp8_linear(codes, scales, dev[2], dev[3])
    assert Y.shape == (0, 40)


def test_refusals(cuda_lib):
    host, (x8, sx, w8, sw) = _quantized(4, 256, 40, seed=1)
    x = _values(4, 256, 0).cuda()
    lin = cuda_lib.fp8_linear
    with pytest.raises(ValueError):
        cuda_lib.fp8_quantize_act(x.t())                         # not contiguous
    with pytest.raises(TypeError):
        cuda_lib.fp8_quantize_act(x.to(torch.int32))
    with pytest.raises(TypeError):
        cuda_lib.fp8_quantize_weight(x.double())
    with pytest.raises(ValueError):
        cuda_lib.fp8_quantize_act(x, out=(x8, sx.t().contiguous()))
    with pytest.raises(cuda_lib.GPTQError) as e:
        cuda_lib.fp8_quantize_act(x[:, :24].contiguous())        # 24 channels
    assert e.value.name == "GPTQ_ERR_ARG"
    for bad in ((x8.view(torch.uint8), sx, w8, sw), (x8, sx.double(), w8, sw),
                (x8, sx, w8.view(torch.uint8), sw)):
        with pytest.raises(TypeError):
            lin(*bad)
    for bad in ((x8, sx.t().contiguous(), w8, sw), (x8, sx, w8[:, :128].contiguous(), sw),
                (x8, sx, w8, sw[:, :1].contiguous()), (x8, sx[:, :3].contiguous(), w8, sw)):
        with pytest.raises(ValueError):
            lin(*bad)
    R = torch.zeros(4, 40, device="cuda")
    with pytest.raises(TypeError):
        lin(x8, sx, w8, sw, R=R)                                 # fp32 residual, fp16 output
    with pytest.raises(TypeError):
        lin(x8, sx, w8, sw, dtype=torch.float64)
    with pytest.raises(ValueError):
        lin(x8, sx, w8, sw, R=R[:, :39], dtype=F32)
    with pytest.raises(TypeError):
        lin(x8, sx, w8, sw, status=R)
