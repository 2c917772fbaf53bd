"""Gradient of the sigmoid balance loss where experts are saturated: relative to itself, also where 1 - sigma is small.

Tolerance (u = 2^-24), for logits that matter of at most L: an exponential e^x of a difference of at most L has
the roundings of the difference, of the product with log2(e) and of that constant, each L u at most, and 2 ulp of its
own: (3 L + 4) u.  A score is a quotient of 1 / (a + y) and its sum, with two exponentials at most, an addition and a
quotient (2 ulp) each, and E / 8 + 5 additions of one sign: P = 2 (6 L + 8 + 6) + E / 8 + 9.  The mean over scores adds as many
additions, 1 - sigma is a quotient of the same quantities, 2 (3 L + 4) + 8, the common factor has 8 roundings and the
products 4."""
import numpy as np
import pytest
import torch

from fp8_fp4_moe_b200 import binding
from oracle import training as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _check(l, ids, L, offsets=None):
    E = l.shape[1]
    k = ids.shape[1]
    do = None if offsets is None else offsets.cuda()
    args = dict(coef=0.01, offsets=do, score="sigmoid")
    loss, counts, probs, tokens = binding.balance_loss(l.cuda(), ids.cuda(), **args)
    grad = binding.balance_loss_backward(torch.tensor(1.5, device="cuda"), l.cuda(), counts, tokens, k, **args)
    o = None if offsets is None else offsets.numpy()
    ref, mag = O.balance_grad(1.5, l.double().numpy(), ids.numpy(), 0.01, o, score="sigmoid")
    P = 2 * (6 * L + 14) + E / 8 + 9
    tol = (2 * P + E / 8 + 5 + 2 * (3 * L + 4) + 8 + 12) * U * mag + 1e-37
    if l.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref)
    got = grad.double().cpu().numpy()
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert bad.size == 0, (len(bad), bad[:4], got[tuple(bad[0])], ref[tuple(bad[0])])
    p = O.balance_loss(l.double().numpy(), ids.numpy(), 0.01, o, score="sigmoid")[2]
    assert (np.abs(probs.cpu().numpy() - p) <= (l.shape[0] + P) * U * p + 1e-37).all()


@pytest.mark.parametrize("E,k", [(3, 1), (8, 2), (48, 4), (256, 8), (257, 3), (600, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_saturated_experts(cuda_lib, E, k, dtype):
    g = torch.Generator().manual_seed(E)
    l = torch.randn(120, E, generator=g)
    sign = torch.where(torch.rand(120, E, generator=g) < 0.5, 1.0, -1.0)
    for i, size in enumerate((4, 9, 16, 20, 25, 30)):
        l[8 * i:8 * i + 4] += size * (torch.rand(4, E, generator=g) < 0.3)       # some far above
        l[8 * i + 4:8 * i + 8] = size * sign[8 * i + 4:8 * i + 8] * torch.rand(4, E, generator=g)
    l = l.clamp(-32, 32).to(dtype)
    ids = torch.topk(torch.rand(120, E, generator=g), k, dim=1).indices.to(torch.int32)
    _check(l, ids, 32)
    _check(l, ids, 32, torch.tensor([0, 50, 50, 119], dtype=torch.int32))


@pytest.mark.parametrize("E", [8, 64, 256])
def test_rows_around_every_size(cuda_lib, E):
    # rows whose largest logit lies anywhere from far below zero, where every sigma underflows, to far above, side by side
    g = torch.Generator().manual_seed(E + 1)
    tops = torch.cat([torch.linspace(-300, 80, 77), torch.tensor([-1e4, -2000.0, -87.5, -88.0, -69.1, 0.0])])
    l = tops[:, None] - 8 * torch.rand(len(tops), E, generator=g)
    l[:, E // 2] = tops
    ids = torch.randint(0, E, (len(tops), 2), generator=g).to(torch.int32)
    perm = torch.randperm(len(tops), generator=g)
    _check(l[perm], ids, 88)


def test_low_logits_beside_a_row_top_below_zero(cuda_lib):
    # sigma of the lower ones is below fp32's normal range, their share of the row is not
    l = torch.full((9, 16), -60.0)
    l[:, 1::2] = -88.0
    l[4, 0] = -59.0
    l[5] = -85.0
    ids = torch.arange(18).remainder(16).reshape(9, 2).to(torch.int32)
    _check(l, ids, 88)
