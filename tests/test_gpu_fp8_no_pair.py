"""Large calls of fp8_linear where its kernel for pairs of CTAs cannot be launched: the streaming
kernel serves them. Small-integer codes and power-of-two scales make every bit of Y determined."""

import pytest
import torch

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.mark.parametrize("n,d_in,d_out,dtype,res", [
    (1500, 1024, 2056, F16, True), (2600, 144, 4104, F32, True), (1030, 128, 2049, BF16, False),
    (5000, 256, 1030, F32, False)])
def test_the_streaming_kernel_serves_large_calls(cuda_lib, n, d_in, d_out, dtype, res):
    g = torch.Generator(device="cuda").manual_seed(n)

    def ints(r, c, hi):
        return torch.randint(-hi, hi + 1, (r, c), generator=g, device="cuda").float()

    nb, no = -(-d_in // 128), -(-d_out // 128)
    ins = (ints(n, d_in, 3).to(E4M3), 2.0 ** ints(nb, n, 2), ints(d_out, d_in, 3).to(E4M3),
           2.0 ** ints(no, nb, 2))
    R = ints(n, d_out, 8).to(dtype) if res else None
    want = cuda_lib.fp8_linear(*ins, R=R, dtype=dtype)
    cuda_lib.test_fp8_no_pair(True)
    try:
        got = cuda_lib.fp8_linear(*ins, R=R, dtype=dtype)
    finally:
        cuda_lib.test_fp8_no_pair(False)
    assert torch.equal(got, want)
    X = ins[0].double() * ins[1].t().repeat_interleave(128, 1)[:, :d_in]
    W = ins[2].double() * (ins[3].repeat_interleave(128, 0)[:d_out].repeat_interleave(128, 1)[:, :d_in])
    ref = X @ W.t() + (R.double() if res else 0.0)
    assert torch.equal(got, ref.float().to(dtype))
