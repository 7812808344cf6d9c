"""Keys near fp16's largest value: the scale is rounded up, so they can read back above it. The
values are scale·(code - zero) rounded once to the output's type, infinite in fp16 from 65520 on."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as okv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,top", [(8, 65535.0), (4, 65520.0)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_largest_keys_read_back(cuda_lib, bits, top, sign):
    H, D, g = 1, 64, 32
    K = torch.zeros(2, H, D, dtype=torch.float16)
    K[0, 0, :g] = sign * torch.linspace(0, 65504, g).half()
    K[1, 0, g:] = sign * torch.linspace(0, 60000, g).half()        # stays below
    dev = cuda_lib.kv_cache_alloc(1, 2, H, D, bits, g)
    host = [t.cpu().numpy() for t in dev]
    cuda_lib.kv_cache_write(K.cuda(), K.cuda(), torch.arange(2, device="cuda"), *dev, bits=bits)
    okv.write(*host, K.double().numpy(), K.double().numpy(), [0, 1], bits)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    ref, _ = okv.read(*host, table.cpu().numpy(), [0, 2], bits)
    assert np.max(np.abs(ref)) == top
    for dtype in (torch.float16, torch.bfloat16, torch.float32):
        k, v = cuda_lib.kv_cache_read(*dev, table, cu, 2, bits=bits, dtype=dtype)
        want = torch.from_numpy(ref).float().to(dtype)
        assert torch.equal(k.cpu(), want) and torch.equal(v.cpu(), want)
        if dtype == torch.float16:
            assert bool(torch.isinf(want).any()) and bool(torch.isfinite(want[1]).all())
        else:
            assert bool(torch.isfinite(want).all())
