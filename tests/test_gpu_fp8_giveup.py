"""fp8_linear when a bounded wait gives up: the call ends by itself and reports GPTQ_ERR_TIMEOUT,
nothing but Y is touched, and the next call is right. The give-up is a host switch that makes one
CTA's producer stop early, with waits of about 1 ms; no fault and no hang is provoked."""

import pytest
import torch

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32
TIMEOUT = -6


def _inputs(n, d_in, d_out):
    g = torch.Generator(device="cuda").manual_seed(n + d_in + d_out)

    def codes(r, c):
        return torch.randint(-3, 4, (r, c), generator=g, device="cuda").float().to(E4M3)

    def scales(r, c):
        return torch.rand(r, c, generator=g, device="cuda") + 0.5

    nb = -(-d_in // 128)
    return codes(n, d_in), scales(nb, n), codes(d_out, d_in), scales(-(-d_out // 128), nb)


def _give_up_and_recover(lib, n, d_in, d_out, rank, dtype, res):
    ins = _inputs(n, d_in, d_out)
    R = torch.ones(n, d_out, dtype=dtype, device="cuda") if res else None
    want = lib.fp8_linear(*ins, R=R, dtype=dtype)
    buf = torch.full((n + 16, d_out), 7.0, dtype=dtype, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    lib.test_stall_fp8(rank)
    try:
        lib.fp8_linear(*ins, R=R, out=buf[8:-8], status=status)
    finally:
        lib.test_stall_fp8(None)
    torch.cuda.synchronize()
    assert int(status) == TIMEOUT
    assert bool((buf[:8] == 7).all()) and bool((buf[-8:] == 7).all())
    status.zero_()
    again = lib.fp8_linear(*ins, R=R, dtype=dtype, status=status)
    assert torch.equal(again, want) and int(status) == 0


@pytest.mark.parametrize("rank", [0, 1, 7])
@pytest.mark.parametrize("n,dtype,res", [(5, F16, True), (20, F32, False), (50, BF16, True), (100, F16, False)])
def test_streaming_call_gives_up_in_a_cluster(cuda_lib, n, dtype, res, rank):
    """d_in is split over eight CTAs, which wait for one another's sums."""
    _give_up_and_recover(cuda_lib, n, 8192, 520, rank, dtype, res)


@pytest.mark.parametrize("n", [5, 50])
def test_streaming_call_gives_up_alone(cuda_lib, n):
    """So many tiles that d_in is not split."""
    _give_up_and_recover(cuda_lib, n, 1024, 296 * 128, 0, F16, True)


@pytest.mark.parametrize("rank", [0, 1])
@pytest.mark.parametrize("n,d_in,d_out,dtype,res", [
    (1500, 2048, 2056, F16, True),       # one tile per pair of CTAs, the residual's copies in flight
    (1500, 2048, 2056, F32, False),
    (1500, 2048, 2051, BF16, True),      # odd rows of Y
    (2600, 256, 4104, F32, True),        # two blocks a tile: the producer stops in its third tile
    (2600, 256, 4104, F16, False),
])
def test_pair_call_gives_up(cuda_lib, n, d_in, d_out, dtype, res, rank):
    """One producer of a pair stops before the other, whose copies are then ahead of it."""
    _give_up_and_recover(cuda_lib, n, d_in, d_out, rank, dtype, res)
