"""Arguments that moe_quant_fp8, moe_gemm_fp8 and the balance loss refuse, before any device work (CPU).
The pointers are made-up addresses: a refused call never reads them."""
import pytest
import torch

from fp8_fp4_moe_b200 import binding, build

ARG, SHAPE, WS = binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_UNSUPPORTED_SHAPE, binding.MOE_ERR_WORKSPACE
P = 0x100000   # an aligned address


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


QUANT = dict(M=4, K=200, x=P, ldx=200, x_type=0, block=0, format=0, scale_type=0, q=P, ldq=208, scales=P, s_row=1,
             s_blk=4, qt=P, ldqt=16, scales_t=P, st_row=1, st_blk=200, stream=None)


@pytest.mark.parametrize("change,code", [
    ({"M": -1}, SHAPE), ({"K": -5}, SHAPE), ({"x_type": 3}, ARG), ({"block": 2}, ARG), ({"format": 2}, ARG),
    ({"scale_type": 2}, ARG), ({"q": None, "qt": None}, ARG), ({"x": None}, ARG), ({"x": P + 1}, ARG), ({"ldx": 199}, ARG),
    ({"q": P + 8}, ARG), ({"ldq": 200}, ARG), ({"ldq": 192}, ARG), ({"scales": None}, ARG), ({"scales": P + 2}, ARG),
    ({"s_row": -1}, ARG), ({"s_blk": -1}, ARG), ({"qt": P + 4}, ARG), ({"ldqt": 8}, ARG), ({"ldqt": 0}, ARG),
    ({"scales_t": None}, ARG), ({"st_row": -1}, ARG), ({"st_blk": -1}, ARG),
    ({"M": 65536 * 128, "ldqt": 65536 * 128}, SHAPE), ({"M": (1 << 30) + 1}, SHAPE), ({"K": (1 << 30) + 1}, SHAPE),
])
def test_quant_refuses(L, change, code):
    assert L.moe_quant_fp8(*(QUANT | change).values()) == code


def test_quant_of_nothing_is_no_launch(L):
    assert L.moe_quant_fp8(*(QUANT | {"M": 0}).values()) == 0
    assert L.moe_quant_fp8(*(QUANT | {"K": 0}).values()) == 0


GEMM = dict(M=4, N=8, K=200, A=P, lda=208, a_format=0, A_scales=P, as_row=1, as_blk=4, a_rows=1, B=P, ldb=208,
            b_format=1, B_scales=P, bs_row=1, bs_blk=1, b_rows=128, scale_type=0, out=P, ldo=8, out_type=0,
            accumulate=0, workspace=P, bytes=256, stream=None)


@pytest.mark.parametrize("change,code", [
    ({"M": (1 << 30) + 1}, SHAPE), ({"N": (1 << 30) + 1}, SHAPE), ({"K": (1 << 28) + 1}, SHAPE),
    ({"M": -1}, SHAPE), ({"N": -1}, SHAPE), ({"K": -1}, SHAPE), ({"a_format": 2}, ARG), ({"b_format": -1}, ARG),
    ({"scale_type": 2}, ARG), ({"out_type": 2}, ARG), ({"accumulate": 1}, ARG), ({"a_rows": 64}, ARG), ({"b_rows": 0}, ARG),
    ({"workspace": None}, WS), ({"workspace": P + 128}, WS), ({"bytes": 255}, WS), ({"out": None}, ARG), ({"out": P + 1}, ARG),
    ({"out": P + 2, "out_type": 1}, ARG), ({"ldo": 7}, ARG), ({"A": None}, ARG), ({"A": P + 8}, ARG), ({"B": P + 1}, ARG),
    ({"lda": 200}, ARG), ({"ldb": 192}, ARG), ({"A_scales": None}, ARG), ({"B_scales": P + 1}, ARG), ({"as_row": -1}, ARG),
    ({"as_blk": -1}, ARG), ({"bs_row": -1}, ARG), ({"bs_blk": -1}, ARG),
])
def test_gemm_refuses(L, change, code):
    assert L.moe_gemm_fp8(*(GEMM | change).values()) == code


LOSS = dict(T=4, E=8, k=2, S=1, logits=P, ldl=8, type=1, ids=P, offsets=None, mask=None, score=0, coef=1.0, loss=P,
            counts=P, probs=P, tokens=P, workspace=P, bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change,code", [
    ({"T": (1 << 30) + 1}, SHAPE), ({"T": -1}, SHAPE), ({"E": 0}, SHAPE), ({"E": 1025, "ldl": 1025}, SHAPE), ({"k": 0}, SHAPE), ({"k": 9}, SHAPE),
    ({"E": 32, "ldl": 32, "k": 17}, SHAPE), ({"S": 0}, SHAPE), ({"S": (1 << 20) + 1, "offsets": P}, SHAPE), ({"type": 2}, ARG),
    ({"score": 2}, ARG), ({"coef": float("nan")}, ARG), ({"coef": float("inf")}, ARG), ({"logits": None}, ARG),
    ({"logits": P + 2}, ARG), ({"ldl": 7}, ARG), ({"ids": None}, ARG), ({"ids": P + 2}, ARG), ({"S": 2}, ARG),
    ({"S": 2, "offsets": P + 1}, ARG), ({"loss": None}, ARG), ({"counts": None}, ARG), ({"probs": P + 2}, ARG),
    ({"tokens": None}, ARG), ({"workspace": None}, WS), ({"workspace": P + 4}, WS), ({"bytes": 100}, WS),
])
def test_balance_loss_refuses(L, change, code):
    assert L.moe_balance_loss(*(LOSS | change).values()) == code


GRAD = dict(T=4, E=8, k=2, S=1, grad_loss=P, logits=P, ldl=8, type=1, counts=P, tokens=P, offsets=None, mask=None,
            score=0, coef=1.0, grad=P, ldg=8, accumulate=0, stream=None)


@pytest.mark.parametrize("change,code", [
    ({"T": -1}, SHAPE), ({"E": 1025}, SHAPE), ({"k": 0}, SHAPE), ({"S": 0}, SHAPE), ({"type": 2}, ARG), ({"score": -1}, ARG),
    ({"coef": float("nan")}, ARG), ({"grad_loss": None}, ARG), ({"logits": None}, ARG), ({"ldl": 4}, ARG), ({"ldg": 4}, ARG),
    ({"counts": None}, ARG), ({"tokens": P + 1}, ARG), ({"S": 3}, ARG), ({"grad": None}, ARG), ({"grad": P + 2}, ARG),
])
def test_balance_loss_backward_refuses(L, change, code):
    assert L.moe_balance_loss_backward(*(GRAD | change).values()) == code


def test_balance_workspace_sizes(L):
    assert L.moe_balance_workspace_bytes(512, 256, 1) > 0
    assert L.moe_balance_workspace_bytes(0, 256, 1) > 0
    for bad in ((-1, 256, 1), (512, 0, 1), (512, 1025, 1), (512, 256, 0), (512, 256, (1 << 20) + 1)):
        assert L.moe_balance_workspace_bytes(*bad) == 0


def test_the_binding_refuses_on_the_host(L):
    f8 = torch.float8_e4m3fn
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.quant_fp8(x)                                    # not a CUDA tensor
    with pytest.raises(ValueError):
        binding.quant_fp8(x[0])
    with pytest.raises(ValueError):
        binding.quant_fp8(x.t())                                # rows not contiguous
    with pytest.raises(ValueError):
        binding.quant_fp8(x, block="column")
    with pytest.raises(ValueError):
        binding.quant_fp8(x, rows=False)
    with pytest.raises(TypeError):
        binding.quant_fp8(x.double())
    with pytest.raises(TypeError):
        binding.quant_fp8(x, dtype=torch.int8)
    with pytest.raises(TypeError):
        binding.quant_fp8(x, scale_dtype=torch.bfloat16)
    a, b = torch.zeros(4, 256, dtype=f8), torch.zeros(8, 256, dtype=f8)
    sa, sb = torch.ones(4, 2), torch.ones(1, 2)
    with pytest.raises(ValueError):
        binding.gemm_fp8(a, sa, b, sb)                          # not CUDA tensors
    with pytest.raises(ValueError):
        binding.gemm_fp8(a, sa, b[:, :128], sb)
    with pytest.raises(ValueError):
        binding.gemm_fp8(a, sa[:, :1], b, sb)
    with pytest.raises(TypeError):
        binding.gemm_fp8(a, sa, b, sb.to(torch.uint8))          # two scale types
    with pytest.raises(TypeError):
        binding.gemm_fp8(a, sa.double(), b, sb.double())
    with pytest.raises(TypeError):
        binding.gemm_fp8(a.to(torch.bfloat16), sa, b, sb)
    with pytest.raises(TypeError):
        binding.gemm_fp8(a, sa, b, sb, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        binding.gemm_fp8(a, sa, b, sb, accumulate=True)
    with pytest.raises(ValueError):
        binding.gemm_fp8(a, sa, b, sb, out=torch.zeros(8, 4))
    l, ids = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError):
        binding.balance_loss(l, ids)                            # not CUDA tensors
    with pytest.raises(ValueError):
        binding.balance_loss(l, ids[:3])
    with pytest.raises(TypeError):
        binding.balance_loss(l, ids.long())
    with pytest.raises(TypeError):
        binding.balance_loss(l.double(), ids)
    with pytest.raises(ValueError):
        binding.balance_loss(l, ids, score="softplus")
    with pytest.raises(ValueError):
        binding.balance_loss(l, ids, mask=torch.ones(3, dtype=torch.bool))
    with pytest.raises(ValueError):
        binding.balance_loss(l, ids, offsets=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(binding.MoeError):
        binding.balance_loss(torch.zeros(2, 1025), torch.zeros(2, 1, dtype=torch.int32))
    c, n, g = torch.zeros(1, 8, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.ones(())
    with pytest.raises(ValueError):
        binding.balance_loss_backward(g, l, c[:, :4], n, 2)
    with pytest.raises(ValueError):
        binding.balance_loss_backward(g, l, c, n, 2, accumulate=True)
    with pytest.raises(TypeError):
        binding.balance_loss_backward(g, l, c, n, 2, out=torch.zeros(4, 8, dtype=torch.bfloat16))
