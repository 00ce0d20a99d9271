"""GPU: the 8-bit quantiser at its largest extents, where offsets pass 32 bits."""
import pytest

import mixed_precision_matmul_gb300 as mpg

pytestmark = pytest.mark.gpu

TOP = 2 ** 31 - 256


@pytest.mark.parametrize("rows,cols", [(1, TOP), (TOP, 1), (TOP - 77, 1)])
def test_quantizer_at_its_largest_extents(rows, cols):
    import torch
    mpg.build()
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("24 GB of device memory are not free")
    n = rows * cols
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    part = torch.randn(1 << 16, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    ends = [slice(0, 1 << 16), slice(1 << 30, (1 << 30) + (1 << 16)), slice(n - (1 << 16) // 128 * 128 - n % 128, n)]
    for e in ends:
        x[e] = torch.cat([part, part])[:e.stop - e.start]
    q = torch.full((n + 64,), 0x55, dtype=torch.uint8, device="cuda")
    blocks = -(-cols // 128)
    s = torch.empty(rows * blocks, device="cuda")
    mpg.fp8_quantize_raw(rows, cols, x.data_ptr(), cols, mpg.BF16, mpg.E4M3, 1, q.data_ptr(), cols, s.data_ptr(), blocks, 1, 0,
                         0, 0, 0, 0)
    torch.cuda.synchronize()
    assert mpg.device_status() == mpg.OK
    for e in ends:
        lines = x[e].view(1, -1) if rows == 1 else x[e].view(-1, 1)
        wq, ws = mpg.fp8_quantize(lines)
        assert torch.equal(q[e].view(torch.float8_e4m3fn).float(), wq.float().flatten())
        first = e.start // 128 if rows == 1 else e.start
        assert torch.equal(s[first:first + ws.numel()], ws.flatten())
    assert (q[n:] == 0x55).all()
    assert not q[1 << 17:(1 << 17) + 4096].any()              # zeros between
