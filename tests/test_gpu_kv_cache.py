"""The quantised key/value cache against the fp64 oracle. Codes, scales and zeros are compared bit
for bit (the quantizer is exact). Read-back values are compared exactly too: scale·(code - zero)
has at most 20 significant bits, so it is exact in fp32 and rounded once to the output type."""

import numpy as np
import pytest
import torch

from oracle import fp8 as ofp8
from oracle import kv_cache as okv

pytestmark = pytest.mark.gpu
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


def _np(t):
    return t.detach().cpu().double().numpy()


def _kv(n, H, D, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    mag = torch.exp(torch.randn(H, D, generator=g))
    return [(torch.randn(n, H, D, generator=g) * mag).to(dtype) for _ in range(2)]


def _filled(lib, n_pages, page, H, D, bits, g, seed):
    """A cache with something in every slot, on the device and on the host."""
    gen = torch.Generator().manual_seed(seed)
    dev = lib.kv_cache_alloc(n_pages, page, H, D, bits, g)
    dev[0].copy_(torch.randint(0, 256, dev[0].shape, generator=gen, dtype=torch.uint8))
    dev[1].copy_(torch.rand(dev[1].shape, generator=gen).to(F16))
    dev[2].copy_(torch.randint(0, 2 ** bits, dev[2].shape, generator=gen).to(F16))
    return dev, [t.cpu().numpy().copy() for t in dev]


def _same(got, ref):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape and np.array_equal(np.isnan(got), np.isnan(ref))
    ok = ~np.isnan(ref)
    assert np.array_equal(got[ok], ref[ok]), int(np.sum(got[ok] != ref[ok]))


def _rounded(x64, dtype):
    """fp64 values that are exact in fp32, rounded once to dtype."""
    f = torch.from_numpy(np.asarray(x64, np.float64)).float()
    return f.to(dtype).double().numpy()


SHAPES = [   # H, D, bits, group, page
    (1, 16, 4, 16, 1), (1, 16, 8, 16, 5), (8, 128, 8, 128, 16), (8, 128, 4, 64, 64),
    (3, 80, 4, 16, 17), (2, 96, 8, 32, 16), (5, 256, 4, 256, 3), (32, 128, 8, 32, 16),
    (1, 64, 4, 64, 16), (7, 160, 8, 32, 2),
]


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("H,D,bits,g,page", SHAPES)
@pytest.mark.parametrize("n", [1, 3, 37])
def test_write_matches_the_oracle(cuda_lib, n, H, D, bits, g, page, dtype):
    """Every code, scale and zero; slots out of order, one skipped, all other slots as they were."""
    n_pages = (n + page - 1) // page + 2
    dev, host = _filled(cuda_lib, n_pages, page, H, D, bits, g, seed=n)
    K, V = _kv(n, H, D, dtype, seed=n + D)
    perm = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(n))[:n]
    if n > 2:
        perm[1] = -1
    cuda_lib.kv_cache_write(K.cuda(), V.cuda(), perm.cuda(), *dev, bits=bits)
    okv.write(*host, _np(K), _np(V), perm.tolist(), bits)
    for d, h in zip(dev, host):
        _same(d.cpu().numpy(), h)


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("H,D,bits,g", [
    (8, 128, 4, 64), (8, 128, 8, 128), (4, 256, 8, 256), (8, 128, 4, 32), (8, 128, 8, 16),
    (4, 128, 4, 128), (4, 128, 8, 32), (4, 128, 4, 16), (2, 128, 4, 64), (3, 80, 8, 16)])
def test_a_long_write_is_many_short_ones(cuda_lib, H, D, bits, g, dtype):
    """Thousands of tokens in one call leave the cache bit for bit as calls of 100 tokens do, and
    those are checked against the oracle above; the last tokens against the oracle here too."""
    page, n = 64, 5003
    n_pages = n // page + 3
    one, host = _filled(cuda_lib, n_pages, page, H, D, bits, g, seed=5)
    many = [t.clone() for t in one]
    K, V = _kv(n, H, D, dtype, seed=D + H)
    K[7, 0, 3], V[n - 2, H - 1, D - 1] = float("nan"), float("inf")
    perm = torch.randperm(n_pages * page, generator=torch.Generator().manual_seed(H))[:n]
    perm[5::50] = -1
    kd, vd, pd = K.cuda(), V.cuda(), perm.cuda()
    cuda_lib.kv_cache_write(kd, vd, pd, *one, bits=bits)
    for i in range(0, n, 100):
        cuda_lib.kv_cache_write(kd[i:i + 100], vd[i:i + 100], pd[i:i + 100], *many, bits=bits)
    for a, b in zip(one, many):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    okv.write(*host, _np(K[-40:]), _np(V[-40:]), perm[-40:].tolist(), bits)
    slots = perm[-40:][perm[-40:] >= 0].numpy()
    for d, h in zip(one, host):
        _same(d.cpu().numpy().reshape(2, n_pages * page, -1)[:, slots],
              h.reshape(2, n_pages * page, -1)[:, slots])


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("H,D,bits,g,page", SHAPES)
def test_read_matches_the_oracle(cuda_lib, H, D, bits, g, page, dtype):
    """Ragged lengths with empty sequences at the start, inside and at the end; pages that end
    inside a sequence's last one."""
    lens = [0, 1, page, page + 1, 0, 0, 3 * page - 1, 2, 0]
    cu = np.cumsum([0] + lens)
    n_pages = sum(-(-x // page) for x in lens) + 1
    dev, host = _filled(cuda_lib, n_pages, page, H, D, bits, g, seed=D)
    ids = np.random.default_rng(D).permutation(n_pages)
    table = np.full((len(lens), 4), -1, np.int32)
    at = 0
    for b, x in enumerate(lens):
        k = -(-x // page)
        table[b, :k] = ids[at:at + k]
        at += k
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    K, V = cuda_lib.kv_cache_read(*dev, torch.from_numpy(table).cuda(),
                                  torch.from_numpy(cu.astype(np.int32)).cuda(), int(cu[-1]),
                                  bits=bits, dtype=dtype, status=status)
    rk, rv = okv.read(*host, table, cu, bits)
    _same(_np(K), _rounded(rk, dtype))
    _same(_np(V), _rounded(rv, dtype))
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("H,D,bits,g", [
    (32, 128, 4, 64), (8, 128, 8, 128), (4, 256, 4, 32), (4, 128, 8, 64), (2, 128, 4, 16),
    (1, 128, 8, 32), (3, 80, 4, 16), (7, 160, 8, 32)])
def test_a_long_read_is_many_short_ones(cuda_lib, H, D, bits, g, dtype):
    """Thousands of ragged tokens in one call give bit for bit what a call per sequence gives, and
    those are checked against the oracle above; one sequence against the oracle here too. Rows
    before the first sequence and behind the last stay as they were."""
    page, rng = 16, np.random.default_rng(H + D)
    lens = rng.integers(0, 1200, 40)
    lens[3], lens[11] = 0, 1
    first, extra = 5, 9
    cu = (first + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
    total = int(cu[-1]) + extra
    n_pages = int(sum(-(-x // page) for x in lens)) + 1
    dev, host = _filled(cuda_lib, n_pages, page, H, D, bits, g, seed=D)
    ids = rng.permutation(n_pages)
    table = np.full((len(lens), 75), -1, np.int32)
    at = 0
    for b, x in enumerate(lens):
        k = -(-int(x) // page)
        table[b, :k] = ids[at:at + k]
        at += k
    K = torch.full((total, H, D), 7.0, dtype=dtype, device="cuda")
    V = torch.full((total, H, D), -7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    td = torch.from_numpy(table).cuda()
    cuda_lib.kv_cache_read(*dev, td, torch.from_numpy(cu).cuda(), total, bits=bits, dtype=dtype,
                           out=(K, V), status=status)
    for b, x in enumerate(lens):
        one = torch.tensor([0, int(x)], dtype=torch.int32, device="cuda")
        k, v = cuda_lib.kv_cache_read(*dev, td[b:b + 1], one, int(x), bits=bits, dtype=dtype)
        assert torch.equal(K[cu[b]:cu[b + 1]], k) and torch.equal(V[cu[b]:cu[b + 1]], v), b
    assert bool((K[:first] == 7).all()) and bool((K[cu[-1]:] == 7).all())
    assert bool((V[:first] == -7).all()) and bool((V[cu[-1]:] == -7).all())
    rk, rv = okv.read(*host, table[5:6], np.array([0, lens[5]]), bits)
    _same(_np(K[cu[5]:cu[6]]), _rounded(rk, dtype))
    _same(_np(V[cu[5]:cu[6]]), _rounded(rv, dtype))
    assert int(status) == 0


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_read_into_rows_at_any_16_bytes(cuda_lib, dtype):
    """Outputs that start 16 bytes behind a 32-byte boundary get the same values."""
    H, D, bits, g, page, n = 4, 128, 8, 64, 16, 333
    dev, _ = _filled(cuda_lib, 21, page, H, D, bits, g, seed=1)
    table = torch.randperm(21, generator=torch.Generator().manual_seed(2)).int().view(1, -1).cuda()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    ref = cuda_lib.kv_cache_read(*dev, table, cu, n, bits=bits, dtype=dtype)
    skip = 16 // ref[0].element_size()
    flat = torch.zeros(2, n * H * D + 2 * skip, dtype=dtype, device="cuda")
    out = tuple(x[skip:skip + n * H * D].view(n, H, D) for x in flat)
    assert all(x.data_ptr() % 16 == 0 for x in out) and out[0].data_ptr() % 32 == 16
    cuda_lib.kv_cache_read(*dev, table, cu, n, bits=bits, out=out)
    for a, b, x in zip(out, ref, flat):
        assert torch.equal(a, b) and not bool(x[:skip].any()) and not bool(x[-skip:].any())


@pytest.mark.parametrize("n_seqs", [1, 2, 31, 32, 33, 64, 1000, 1025, 2500])
def test_read_finds_every_sequence(cuda_lib, n_seqs):
    """Rows of many sequences, some empty: each row comes from its own sequence's page."""
    H, D, bits, g, page = 1, 16, 8, 16, 2
    rng = np.random.default_rng(n_seqs)
    lens = rng.integers(0, 5, n_seqs)
    lens[rng.integers(0, n_seqs)] = 2
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n_pages = 3 * n_seqs
    dev = cuda_lib.kv_cache_alloc(n_pages, page, H, D, bits, g)
    page_id = torch.arange(n_pages, device="cuda")
    dev[1].fill_(1.0)                                  # value = code - zero = code
    dev[0][0] = (page_id % 251).to(torch.uint8).view(-1, 1, 1, 1)
    dev[0][1] = (page_id // 251).to(torch.uint8).view(-1, 1, 1, 1)
    table = rng.permutation(n_pages).reshape(n_seqs, 3)[:, :2].astype(np.int32)
    total = int(cu[-1])
    K, V = cuda_lib.kv_cache_read(*dev, torch.from_numpy(table).cuda(),
                                  torch.from_numpy(cu).cuda(), total, bits=bits)
    got = (K + 251 * V.float()).cpu().numpy()
    seq = np.repeat(np.arange(n_seqs), lens)
    pos = np.arange(total) - cu[seq]
    want = table[seq, pos // page]
    assert np.array_equal(got, np.broadcast_to(want[:, None, None], got.shape))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("dtype", [F16, BF16, F32])
def test_edge_groups(cuda_lib, dtype, bits):
    """Zero groups, one-sided groups, the type's largest and smallest values, ties, NaN and
    infinities; what is not finite stays in its own group and reads back as NaN."""
    H, D, g, page = 1, 128, 32, 4
    fi = torch.finfo(dtype)
    K, V = _kv(12, H, D, dtype, seed=1)
    K[0] = 0.0
    K[1] = -0.0
    K[2] = K[2].abs() + 1
    K[3] = -K[3].abs() - 1
    K[4] = 5.0
    K[5, 0, 0], K[5, 0, 1] = fi.max, -fi.max
    K[6] = fi.smallest_normal * fi.eps
    K[7, 0, 40] = float("nan")
    K[8, 0, 70] = float("inf")
    K[9, 0, 127] = -float("inf")
    K[10, 0, :] = torch.arange(128).to(dtype) / 2          # many exact ties
    V[11] = float("nan")
    dev = cuda_lib.kv_cache_alloc(3, page, H, D, bits, g)
    host = [t.cpu().numpy() for t in dev]
    slots = torch.arange(12)
    cuda_lib.kv_cache_write(K.cuda(), V.cuda(), slots.cuda(), *dev, bits=bits)
    okv.write(*host, _np(K), _np(V), slots.tolist(), bits)
    for d, h in zip(dev, host):
        _same(d.cpu().numpy(), h)
    table = torch.tensor([[0, 1, 2]], dtype=torch.int32)
    cu = torch.tensor([0, 12], dtype=torch.int32)
    k, v = cuda_lib.kv_cache_read(*dev, table.cuda(), cu.cuda(), 12, bits=bits, dtype=dtype)
    rk, rv = okv.read(*host, table.numpy(), [0, 12], bits)
    _same(_np(k), _rounded(rk, dtype))
    _same(_np(v), _rounded(rv, dtype))
    assert bool(torch.isnan(v[11]).all()) and bool(torch.isnan(k[7, 0, 32:64]).all())
    assert not bool(torch.isnan(k[7, 0, :32]).any())


def test_write_takes_views_of_a_fused_projection(cuda_lib):
    """Keys and values as column ranges of [n, q;k;v] rows, and keys shared by broadcast."""
    n, H, D, bits, g, page = 19, 4, 64, 4, 32, 8
    qkv = torch.randn(n, 3 * H * D, generator=torch.Generator().manual_seed(1)).to(F16).cuda()
    K = qkv[:, H * D:2 * H * D].unflatten(1, (H, D))
    V = qkv[:, 2 * H * D:].unflatten(1, (H, D))
    one = K[:1].expand(n, H, D)
    for k in (K, one):
        dev, host = _filled(cuda_lib, 3, page, H, D, bits, g, seed=3)
        slots = torch.arange(n - 1, -1, -1)
        cuda_lib.kv_cache_write(k, V, slots.cuda(), *dev, bits=bits)
        okv.write(*host, _np(k), _np(V), slots.tolist(), bits)
        for d, h in zip(dev, host):
            _same(d.cpu().numpy(), h)


def test_slots_and_pages_outside_the_cache(cuda_lib):
    """A slot behind the cache is skipped, a page outside it or a position behind the table reads
    as zeros; both are reported, everything else is served, and nothing else is touched."""
    H, D, bits, g, page, n_pages = 2, 32, 8, 16, 4, 3
    dev, host = _filled(cuda_lib, n_pages, page, H, D, bits, g, seed=4)
    K, V = _kv(4, H, D, F16, seed=4)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, n_pages * page, -3, 2 ** 62])
    cuda_lib.kv_cache_write(K.cuda(), V.cuda(), slots.cuda(), *dev, bits=bits, status=status)
    okv.write(*host, _np(K), _np(V), slots.tolist(), bits)
    for d, h in zip(dev, host):
        _same(d.cpu().numpy(), h)
    assert int(status) == -1
    status.zero_()
    table = torch.tensor([[2, 0], [3, 1], [1, -1], [0, 2]], dtype=torch.int32)
    cu = torch.tensor([0, 6, 14, 20, 29], dtype=torch.int32)      # the last: 9 of 8 positions
    k, v = cuda_lib.kv_cache_read(*dev, table.cuda(), cu.cuda(), 29, bits=bits, status=status)
    assert int(status) == -1
    bad = np.zeros(29, bool)
    bad[6:10] = True                                              # page 3 of 3
    bad[18:20] = True                                             # page -1
    bad[28] = True                                                # behind the table
    safe = np.where((table.numpy() < 0) | (table.numpy() >= n_pages), 0, table.numpy())
    safe = np.concatenate([safe, np.zeros((4, 1), np.int64)], 1)
    for got, ref in zip((k, v), okv.read(*host, safe, cu.tolist(), bits)):
        ref[bad] = 0.0
        _same(_np(got), _rounded(ref, F16))


def test_rows_of_no_sequence_are_left_as_they_were(cuda_lib):
    H, D, bits, g, page = 2, 32, 4, 32, 4
    dev, host = _filled(cuda_lib, 4, page, H, D, bits, g, seed=5)
    table = torch.tensor([[3, 1], [0, 2]], dtype=torch.int32)
    cu = torch.tensor([2, 8, 11], dtype=torch.int32)
    out = (torch.full((16, H, D), 7.5, dtype=BF16, device="cuda"),
           torch.full((16, H, D), -7.5, dtype=BF16, device="cuda"))
    k, v = cuda_lib.kv_cache_read(*dev, table.cuda(), cu.cuda(), 16, bits=bits, out=out)
    for got, ref, old in zip((k, v), okv.read(*host, table.numpy(), [0, 6, 9], bits), (7.5, -7.5)):
        _same(_np(got[2:11]), _rounded(ref, BF16))
        assert bool((got[:2] == old).all()) and bool((got[11:] == old).all())


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^32 bytes (and values plane): its first and last slots."""
    H, D, bits, g, page = 16, 128, 8, 128, 64
    n_pages = (1 << 32) // (page * H * D) // 2 + 600      # two planes of over 2.1 GB
    codes, scales, zeros = cuda_lib.kv_cache_alloc(n_pages, page, H, D, bits, g)
    assert codes.numel() > 1 << 32
    K, V = _kv(4, H, D, F16, seed=6)
    last = n_pages * page - 1
    slots = torch.tensor([last, 0, last - page, 1])
    cuda_lib.kv_cache_write(K.cuda(), V.cuda(), slots.cuda(), codes, scales, zeros, bits=bits)
    q, s, z = okv.quantize(_np(V), bits, g)
    flat = codes.view(2, n_pages * page, H, D)
    for t in range(4):
        assert np.array_equal(flat[1, int(slots[t])].cpu().numpy(), q[t])
    assert int(torch.count_nonzero(codes)) == int(torch.count_nonzero(
        flat[:, slots.cuda()]))                            # nothing anywhere else
    table = torch.tensor([[n_pages - 2, n_pages - 1]], dtype=torch.int32)
    cu = torch.tensor([0, 2 * page], dtype=torch.int32)
    k, v = cuda_lib.kv_cache_read(codes, scales, zeros, table.cuda(), cu.cuda(), 2 * page, bits=bits)
    _same(_np(v[-1]), _rounded(np.repeat(s[0], g, -1) * (q[0] - np.repeat(z[0], g, -1)), F16))
    q, s, z = okv.quantize(_np(K), bits, g)
    _same(_np(k[page - 1]), _rounded(np.repeat(s[2], g, -1) * (q[2] - np.repeat(z[2], g, -1)), F16))


def test_layer_into_the_cache_and_back(cuda_lib):
    """The run of a served layer: norm, e4m3 activations, the q;k;v projection, keys and values
    into the cache (a prompt, then single tokens, the steps captured in a graph), the context back.
    Each stage is compared with the oracle on the stage's own inputs."""
    d, H, D, bits, g, page, n_seq = 256, 2, 64, 4, 32, 4, 3
    gen = torch.Generator().manual_seed(11)
    W = (0.05 * torch.randn(3 * H * D, d, generator=gen)).to(F16)
    w8, sw = cuda_lib.fp8_quantize_weight(W.cuda())
    dev = cuda_lib.kv_cache_alloc(12, page, H, D, bits, g)
    host = [t.cpu().numpy() for t in dev]
    table = torch.tensor([[5, 0, 9], [2, 7, 1], [11, 3, 4]], dtype=torch.int32)
    lens = [5, 0, 8]

    x8 = torch.empty(n_seq, d, dtype=torch.float8_e4m3fn, device="cuda")
    sx = torch.empty(2, n_seq, device="cuda")
    qkv1 = torch.empty(n_seq, 3 * H * D, dtype=F16, device="cuda")
    X1 = torch.zeros(n_seq, d, dtype=F16, device="cuda")
    slots1 = torch.full((n_seq,), -1, dtype=torch.int64, device="cuda")

    def kv_of(qkv):
        return (qkv[:, H * D:2 * H * D].unflatten(1, (H, D)), qkv[:, 2 * H * D:].unflatten(1, (H, D)))

    def step():
        cuda_lib.fp8_quantize_act(cuda_lib.rms_norm(X1), out=(x8, sx))
        cuda_lib.fp8_linear(x8, sx, w8, sw, out=qkv1)
        cuda_lib.kv_cache_write(*kv_of(qkv1), slots1, *dev, bits=bits)

    # the prompts
    n = sum(lens)
    X = torch.randn(n, d, generator=gen).to(F16).cuda()
    N = cuda_lib.rms_norm(X)
    p8, ps = cuda_lib.fp8_quantize_act(N)
    qkv = cuda_lib.fp8_linear(p8, ps, w8, sw)
    rc, rs = ofp8.quantize_act(_np(N))
    _same(_np(p8), rc)
    ref, mag = ofp8.linear(rc, rs, *ofp8.quantize_weight(_np(W)))
    tol = (4 * 33 * 2.0 ** -23 + 20 * 2.0 ** -24) * mag
    assert np.all(np.abs(_np(qkv) - ref) <= tol + 2.0 ** -11 * (np.abs(ref) + tol) + 2.0 ** -25)
    slot = [int(table[b, p // page]) * page + p % page for b in range(n_seq) for p in range(lens[b])]
    cuda_lib.kv_cache_write(*kv_of(qkv), torch.tensor(slot).cuda(), *dev, bits=bits)
    okv.write(*host, *[_np(t) for t in kv_of(qkv)], slot, bits)

    # single tokens, from a graph
    step()                                            # all slots skipped: warms up, writes nothing
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        X1.copy_(torch.randn(n_seq, d, generator=gen).to(F16))
        slot = [int(table[b, lens[b] // page]) * page + lens[b] % page for b in range(n_seq)]
        slots1.copy_(torch.tensor(slot))
        graph.replay()
        okv.write(*host, *[_np(t) for t in kv_of(qkv1)], slot, bits)
        lens = [x + 1 for x in lens]
    for a, h in zip(dev, host):
        _same(a.cpu().numpy(), h)
    cu = np.cumsum([0] + lens).astype(np.int32)
    k, v = cuda_lib.kv_cache_read(*dev, table.cuda(), torch.from_numpy(cu).cuda(), int(cu[-1]), bits=bits)
    for got, r in zip((k, v), okv.read(*host, table.numpy(), cu, bits)):
        _same(_np(got), _rounded(r, F16))


def test_empty_calls(cuda_lib):
    dev = cuda_lib.kv_cache_alloc(2, 4, 2, 32, 8, 16)
    K = torch.empty(0, 2, 32, dtype=F16, device="cuda")
    cuda_lib.kv_cache_write(K, K, torch.empty(0, dtype=torch.int64, device="cuda"), *dev)
    k, v = cuda_lib.kv_cache_read(*dev, torch.empty(0, 3, dtype=torch.int32, device="cuda"),
                                  torch.zeros(1, dtype=torch.int32, device="cuda"), 0)
    assert k.shape == v.shape == (0, 2, 32) and not bool(dev[0].any())
    out = (torch.ones(3, 2, 32, device="cuda"), torch.ones(3, 2, 32, device="cuda"))
    cuda_lib.kv_cache_read(*dev, torch.zeros(2, 1, dtype=torch.int32, device="cuda"),
                           torch.zeros(3, dtype=torch.int32, device="cuda"), 3, out=out)
    assert bool((out[0] == 1).all()) and bool((out[1] == 1).all())


def test_refusals(cuda_lib):
    codes, scales, zeros = cuda_lib.kv_cache_alloc(2, 4, 2, 32, 8, 16)
    K = torch.zeros(3, 2, 32, dtype=F16, device="cuda")
    slots = torch.arange(3, device="cuda")
    table = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    write, read = cuda_lib.kv_cache_write, cuda_lib.kv_cache_read
    cache = (codes, scales, zeros)
    for args in ((K.transpose(1, 2), K, slots, *cache), (K, K[:2], slots, *cache),
                 (K, K.float(), slots, *cache), (K, K, slots[:2], *cache),
                 (K[:, :1], K[:, :1], slots, *cache), (K, K, slots, codes, scales[..., :1], zeros),
                 (K, K, slots, codes[0], scales, zeros), (K, K, slots.cpu(), *cache)):
        with pytest.raises(ValueError):
            write(*args)
    for args in ((K, K, slots.int(), *cache), (K.int(), K.int(), slots, *cache),
                 (K, K, slots, codes.short(), scales, zeros), (K, K, slots, codes, scales.float(), zeros)):
        with pytest.raises(TypeError):
            write(*args)
    with pytest.raises(ValueError):
        write(K, K, slots, *cache, bits=3)
    with pytest.raises(ValueError):
        read(*cache, table, cu[:1], 3)
    with pytest.raises(TypeError):
        read(*cache, table.long(), cu, 3)
    with pytest.raises(TypeError):
        read(*cache, table, cu, 3, dtype=torch.float64)
    with pytest.raises(ValueError):
        read(*cache, table, cu, 3, out=(K[:2], K[:2]))
    odd = torch.zeros(3, 65, dtype=F16, device="cuda")[:, 1:].unflatten(1, (2, 32))
    with pytest.raises(cuda_lib.GPTQError) as e:
        write(odd, odd, slots, *cache)                            # rows at odd addresses
    assert e.value.name == "GPTQ_ERR_ARG"
    with pytest.raises(ValueError):
        cuda_lib.kv_cache_alloc(2, 4, 2, 32, 8, 24)
