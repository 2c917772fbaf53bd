"""Block quantisation (moe_quant_fp8) against the float64 definition: codes and scales bit for bit, at sizes
that end inside a block, for every input type, format, block and direction."""
import numpy as np
import pytest
import torch

from fp8_fp4_moe_b200 import binding
from oracle import training as O

pytestmark = pytest.mark.gpu

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _x(seed, M, K, dtype):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(2 * torch.randn(M, K, generator=g))
    x *= torch.exp2(torch.randint(-10, 4, (M, 1), generator=g).float())
    x[torch.rand(M, K, generator=g) < 0.05] = 0
    x[torch.rand(M, K, generator=g) < 0.01] = -0.0
    return x.to(dtype)


def _scales(p, scale_dtype):
    return (p + 127).astype(np.uint8) if scale_dtype == torch.uint8 else np.exp2(p.astype(np.float64)).astype(np.float32)


def _check(x, fmt, block, rows, cols, scale_dtype, **kw):
    q, s, qt, st = binding.quant_fp8(x, block=block, rows=rows, cols=cols, dtype=FP8[fmt], scale_dtype=scale_dtype, **kw)
    v = x.double().cpu().numpy()
    for want, codes, scales, m in ((rows, q, s, v), (cols, qt, st, v.T)):
        if not want:
            assert codes is None and scales is None
            continue
        ref, p = O.quant(m, block, fmt)
        got = codes.view(torch.uint8).cpu().numpy()
        nan = np.isnan(m)
        np.testing.assert_array_equal(got[~nan], ref[~nan])
        assert np.isnan(O.decode_fp8(got[nan], fmt)).all()
        np.testing.assert_array_equal(scales.cpu().numpy(), _scales(p, scale_dtype))
        assert scales.dtype == scale_dtype and codes.dtype == FP8[fmt]
        assert codes.shape[0] == 1 or codes.stride(0) % 16 == 0


@pytest.mark.parametrize("M,K", [(1, 1), (1, 128), (1, 7168), (3, 16), (5, 129), (16, 300), (127, 127), (128, 128),
                                 (129, 257), (200, 1000), (64, 2048)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_rows(cuda_lib, M, K, dtype):
    _check(_x(M + K, M, K, dtype).cuda(), "e4m3", "row", True, False, torch.float32)


@pytest.mark.parametrize("M,K", [(1, 1), (1, 300), (7, 128), (130, 40), (128, 256), (257, 129), (300, 520)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("rows", [True, False])
def test_both_directions(cuda_lib, M, K, dtype, block, rows):
    _check(_x(M * 3 + K, M, K, dtype).cuda(), "e4m3", block, rows, True, torch.uint8)


@pytest.mark.parametrize("block", ["row", "tile"])
@pytest.mark.parametrize("scale_dtype", [torch.float32, torch.uint8])
def test_e5m2(cuda_lib, block, scale_dtype):
    _check(_x(9, 140, 210, torch.bfloat16).cuda(), "e5m2", block, True, True, scale_dtype)
    _check(_x(8, 33, 400, torch.float32).cuda(), "e5m2", block, True, False, scale_dtype)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block,cols", [("row", False), ("row", True), ("tile", True)])
def test_special_values(cuda_lib, fmt, block, cols):
    top = O.FORMATS[fmt][2]
    x = _x(4, 140, 520, torch.float32)
    x[0] = 0                                             # empty blocks
    x[:, 130] = 0
    x[1, :128] = top * 2.0 ** torch.arange(-60, 68).float()
    x[2, 5] = float("nan")
    x[3, 200] = float("inf")
    x[4, 300] = -float("inf")
    x[5, :] = torch.finfo(torch.float32).tiny * 2.0 ** -20   # subnormal inputs
    x[6, :] = torch.finfo(torch.float32).max
    x[7, :] = torch.finfo(torch.float32).min
    x[8, :] = float("nan")
    x[9, 0] = top                                        # exactly the largest value at scale 1
    x[9, 1:128] = 0.25
    _check(x.cuda(), fmt, block, True, cols, torch.uint8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block,cols", [("row", False), ("row", True), ("tile", True)])
def test_special_16_bit_values(cuda_lib, dtype, fmt, block, cols):
    i = torch.finfo(dtype)
    x = _x(5, 140, 390, dtype)
    x[0, :] = float("nan")
    x[1, 7] = float("nan")
    x[2, 130:140] = float("inf")
    x[3, 200] = -float("inf")
    x[4] = i.max
    x[5] = i.min
    x[6] = i.tiny
    x[7] = i.tiny * 2.0 ** -6                            # subnormal
    x[8] = i.smallest_normal * i.eps
    x[9, 1:] = 0
    x[10] = -0.0
    x[:, 300] = float("nan")
    x[:, 301] = 0
    _check(x.cuda(), fmt, block, True, cols, torch.float32)


def test_every_bf16_value_against_its_block(cuda_lib):
    # all finite bf16 values, each beside an amax that sets the scale: ties and the subnormal codes
    v = torch.arange(0, 0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[(v.float() >= 2.0 ** -40) & (v.float() <= 2.0 ** 40)]
    v = v[: v.numel() // 127 * 127].view(-1, 127)
    x = torch.cat([v, v.float().amax(1, keepdim=True).to(torch.bfloat16) * 16], 1)
    _check(x.cuda(), "e4m3", "row", True, False, torch.float32)
    _check(-x.t().contiguous().cuda(), "e4m3", "row", False, True, torch.float32)


def test_strides_alignment_and_given_outputs(cuda_lib):
    big = _x(11, 150, 420, torch.bfloat16).cuda()
    for x in (big[:, 1:390], big[3:, 8:408], big[::2, :129], big[:, 2:3]):
        _check(x, "e4m3", "row", True, False, torch.float32)
        _check(x, "e4m3", "row", True, True, torch.float32)
        _check(x, "e4m3", "tile", True, True, torch.uint8)
    # caller's buffers: only the codes of the matrix are written, row-major scales are accepted
    x = big[:, :300]
    q = torch.full((152, 320), 0x55, dtype=torch.uint8, device="cuda").view(FP8["e4m3"])
    qt = torch.full((300, 160), 0x55, dtype=torch.uint8, device="cuda").view(FP8["e4m3"])
    s = torch.full((150, 3), -1.0, device="cuda")
    st = torch.full((300, 2), -1.0, device="cuda")
    out = (q[:150, :300], s, qt[:, :150], st)
    _check(x, "e4m3", "row", True, True, torch.float32, out=out)
    assert (q.view(torch.uint8)[150:] == 0x55).all() and (q.view(torch.uint8)[:, 300:] == 0x55).all()
    assert (qt.view(torch.uint8)[:, 150:] == 0x55).all()


def test_empty(cuda_lib):
    for shape in ((0, 256), (5, 0)):
        q, s, qt, st = binding.quant_fp8(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), cols=True)
        assert q.shape == shape and qt.shape == shape[::-1]
        assert s.shape == (shape[0], -(-shape[1] // 128)) and st.shape == (shape[1], -(-shape[0] // 128))


def test_other_stream_and_graph(cuda_lib):
    x = _x(12, 70, 512, torch.bfloat16).cuda()
    want = binding.quant_fp8(x, cols=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = binding.quant_fp8(x, cols=True, stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a.float(), b.float())
    buf = x.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = binding.quant_fp8(buf, cols=True)
    buf.copy_(_x(13, 70, 512, torch.bfloat16).cuda())
    g.replay()
    want = binding.quant_fp8(buf, cols=True)
    for a, b in zip(want, got):
        assert torch.equal(a.float(), b.float())


@pytest.mark.parametrize("block", ["row", "tile"])
def test_offsets_beyond_32_bits(cuda_lib, block):
    """More than 2^31 elements: the last rows, and the last columns of the transposed copy, are those of the rows alone."""
    M, K, tail = 66048, 32776, 384                        # tail starts a row block of the transposed copy
    x = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
    x.normal_()
    q, s, qt, st = binding.quant_fp8(x, block=block, rows=True, cols=True)
    want = binding.quant_fp8(x[-tail:], block=block, rows=True, cols=True)
    n = tail if block == "row" else tail // 128
    assert torch.equal(q[-tail:].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(s[-n:], want[1])
    assert torch.equal(qt[:, -tail:].view(torch.uint8), want[2].view(torch.uint8)) and torch.equal(st[:, -3:], want[3])
    del qt, st
    if block == "row":
        only, so, _, _ = binding.quant_fp8(x)
        assert torch.equal(only.view(torch.uint8), q.view(torch.uint8)) and torch.equal(so, s)
