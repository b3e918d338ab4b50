"""The head-pair forward back to back: many launches in a row, with nothing between them and with a write larger
than L2 between them, so that a launch's first x tiles arrive late. Every launch writes the same bits.

Its loader once armed a slot's barrier for the third task before the first task's x had to have landed.
"""
import pytest
import torch

from state_space_sequence_chunked_b200 import _binding as ssd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(4, 8192, 80, 64, 1, 128), (8, 640, 40, 64, 1, 128)], ids=str)
@pytest.mark.parametrize("flush", [False, True])
def test_back_to_back(cuda_device, shape, flush):
    B, L, H, P, G, N = shape
    r = torch.Generator(device=cuda_device).manual_seed(1)
    x = torch.randn(B, L, H, P, generator=r, device=cuda_device).bfloat16()
    dt = torch.nn.functional.softplus(torch.randn(B, L, H, generator=r, device=cuda_device) - 3).bfloat16()
    Bm, Cm = (torch.randn(B, L, G, N, generator=r, device=cuda_device).bfloat16() for _ in range(2))
    A, D = -torch.rand(H, generator=r, device=cuda_device) - 0.5, torch.ones(H, device=cuda_device)
    assert ssd.fwd_plan(B, L, H, P, G, N, ssd.SSD_BF16, 256)["path"] == "tcgen05"
    call = lambda **k: ssd.ssd_fwd(x, dt, A, Bm, Cm, D, None, chunk=256, **k)  # noqa: E731
    y0, h0 = call()
    torch.cuda.synchronize()
    big = torch.empty(256 << 20, dtype=torch.uint8, device=cuda_device)
    y, h = torch.empty_like(y0), torch.empty_like(h0)
    for _ in range(60):
        if flush:
            big.zero_()
        call(y=y, h_final=h)
    torch.cuda.synchronize()
    assert torch.equal(y.view(torch.uint8), y0.view(torch.uint8)) and torch.equal(h, h0)
