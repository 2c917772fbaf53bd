"""moe_quant_fp8 refuses scale arrays in which two blocks would share a place (CPU: a refused call reads no pointer; an
accepted one would launch, so those are in the GPU test below)."""
import pytest
import torch

from fp8_fp4_moe_b200 import binding, build

ARG = binding.MOE_ERR_INVALID_ARG
P = 0x100000   # an aligned address
QUANT = dict(M=4, K=500, x=P, ldx=500, x_type=0, block=0, format=0, scale_type=0, q=P, ldq=512, scales=P, s_row=1,
             s_blk=4, qt=P, ldqt=16, scales_t=P, st_row=1, st_blk=500, stream=None)


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


@pytest.mark.parametrize("change", [
    {"s_row": 0}, {"s_blk": 0}, {"s_row": 0, "s_blk": 0},            # broadcast
    {"s_blk": 3}, {"s_row": 4, "s_blk": 4}, {"s_row": 3, "s_blk": 1}, {"s_row": 2, "s_blk": 4},
    {"st_row": 0}, {"M": 300, "ldqt": 304, "s_blk": 300, "st_blk": 0}, {"M": 300, "ldqt": 304, "s_blk": 300, "st_blk": 499},
    {"block": 1, "M": 300, "ldqt": 304, "s_blk": 2}, {"block": 1, "M": 300, "ldqt": 304, "s_blk": 3, "st_blk": 3},
])
def test_shared_places_are_refused(L, change):
    assert L.moe_quant_fp8(*(QUANT | change).values()) == ARG


@pytest.mark.gpu
@pytest.mark.parametrize("M,K,strides", [(4, 500, (1, 4)), (4, 500, (4, 1)), (4, 500, (9, 2)), (4, 500, (2, 7)), (1, 500, (0, 1)),
                                         (4, 100, (1, 0)), (1, 100, (0, 0)), (300, 500, (1, 1000))])
def test_places_of_their_own_are_written(cuda_lib, M, K, strides):
    x = torch.randn(M, K, device="cuda") * torch.exp(3 * torch.randn(M, 1, device="cuda"))
    want, ws, _, _ = binding.quant_fp8(x)
    room = torch.full((strides[0] * M + strides[1] * 4 + 1,), -1.0, device="cuda")
    s = room.as_strided((M, -(-K // 128)), strides)
    q = torch.empty(M, 512, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :K]
    got = binding.quant_fp8(x, out=(q, s, None, None))
    assert torch.equal(got[0].view(torch.uint8), want.view(torch.uint8)) and torch.equal(s, ws)
    assert int((room != -1).sum()) == s.numel()


@pytest.mark.gpu
def test_expanded_scales_are_refused(cuda_lib):
    x = torch.randn(8, 256, device="cuda")
    q = torch.empty(8, 256, dtype=torch.float8_e4m3fn, device="cuda")
    for s in (torch.ones(1, 1, device="cuda").expand(8, 2), torch.ones(8, 1, device="cuda").expand(8, 2)):
        with pytest.raises(binding.MoeError):
            binding.quant_fp8(x, out=(q, s, None, None))
        assert (s == 1).all()
