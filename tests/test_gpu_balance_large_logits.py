"""Balance loss and its gradient where a row's largest logit is far from zero.

The tolerances are those of the ordinary rows (tests/test_gpu_balance.py), u = 2^-24: a score is off by at most 112 u as
long as the differences to the row's largest logit are at most 32 or so large that both sides give zero, and every row
here is built that way, from logits that the type holds exactly."""
import numpy as np
import pytest
import torch

from fp8_fp4_moe_b200 import binding
from oracle import training as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SIZES = [3e5, 1e6, 2e6, 1e7, 1e9, 5e9, 1e10, 1e12, 1e20, 1e30, 1.5e38]


def _rows(E, dtype):
    """Rows with a common large value, with one such value among ordinary ones, and with steps beside it."""
    g = torch.Generator().manual_seed(E)
    rows = []
    for size in SIZES:
        for big in (-size, size):
            big = torch.tensor(big).to(dtype).float().item()
            rows.append(torch.full((E,), big))
            one = torch.randn(E, generator=g)
            one[E // 3] = big
            rows.append(one)
            rows.append(torch.where(torch.arange(E) % 2 == 0, torch.tensor(big), torch.tensor(float("-inf"))))
            if size <= 1e7 and dtype == torch.float32:                  # whole steps are exact up to 2^24
                rows.append(round(big) + torch.randint(-12, 12, (E,), generator=g).float())
            rows.append(torch.randn(E, generator=g))                    # an ordinary row beside them
    return torch.stack(rows).to(dtype)


def _both(l, ids, score):
    args = dict(coef=0.01, score=score)
    loss, counts, probs, tokens = binding.balance_loss(l.cuda(), ids.cuda(), **args)
    grad = binding.balance_loss_backward(torch.tensor(1.5, device="cuda"), l.cuda(), counts, tokens, ids.shape[1], **args)
    return loss, counts, probs, tokens, grad


@pytest.mark.parametrize("E", [8, 48, 256, 300])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("repeat", [1, 40])      # one launch, and the partial sums of many blocks
def test_rows_of_large_finite_logits(cuda_lib, E, score, dtype, repeat):
    l = _rows(E, dtype).repeat(repeat, 1)
    T, k = l.shape[0], 2
    ids = torch.stack([torch.arange(T) % E, (torch.arange(T) * 5 + 1) % E], 1).to(torch.int32)
    loss, counts, probs, tokens, grad = _both(l, ids, score)
    v = l.double().numpy()
    ref_loss, ref_c, ref_p, ref_n, _ = O.balance_loss(v, ids.numpy(), 0.01, score=score)
    ref_g, mag = O.balance_grad(1.5, v, ids.numpy(), 0.01, score=score)
    np.testing.assert_array_equal(counts.cpu().numpy(), ref_c)
    rel = (T + 114) * U
    assert (np.abs(probs.cpu().numpy() - ref_p) <= rel * ref_p + 1e-37).all()
    assert abs(loss.item() - ref_loss) <= (rel + 2 * U) * abs(ref_loss)
    tol = 300 * U * mag + 1e-37
    if score == "sigmoid":                       # 1 - sigma to 8 u of 1
        f = np.exp(-np.maximum(v, 0) - np.log1p(np.exp(-np.abs(v))))
        p = O.scores(v, score)
        c = ref_c[0].astype(np.float64)
        whole = 1.5 * 0.01 * E / (k * T) / T * p * (c + (p * c).sum(1, keepdims=True))
        assert np.allclose(whole * f, mag, rtol=1e-12, atol=0)
        tol = tol + 8 * U * whole
    if dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref_g)
    bad = np.argwhere(~(np.abs(grad.double().cpu().numpy() - ref_g) <= tol))
    assert bad.size == 0, (bad[:4], grad[tuple(bad[0])].item(), ref_g[tuple(bad[0])])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("fill", [-1e10, -1e30])
def test_a_masked_out_row_is_even(cuda_lib, score, fill):
    # a usual way to leave a row nothing: every expert at a large negative value; each has the score 1 / E
    l = torch.randn(50, 64, generator=torch.Generator().manual_seed(1))
    l[17] = fill
    ids = torch.zeros(50, 1, dtype=torch.int32)
    off = torch.tensor([0, 17, 18, 50], dtype=torch.int32, device="cuda")
    loss, counts, probs, tokens = binding.balance_loss(l.cuda(), ids.cuda(), offsets=off, score=score)
    assert torch.isfinite(loss) and torch.isfinite(probs).all()
    assert ((probs[1] - 1 / 64).abs() <= 114 * U / 64).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_captured_step_follows_its_logits(cuda_lib, score):
    # ordinary rows in one replay, rows far from zero in the next; padding behind the last sequence stays zero
    E, k = 48, 2
    far = _rows(E, torch.float32)
    T = far.shape[0]
    near = torch.randn(T, E, generator=torch.Generator().manual_seed(3))
    l, ids = near.cuda(), (torch.arange(T * k).reshape(T, k) * 7 % E).to(torch.int32).cuda()
    off = torch.tensor([0, 9, 9, T - 3], dtype=torch.int32, device="cuda")
    one = torch.ones((), device="cuda")

    def step():
        r = binding.balance_loss(l, ids, offsets=off, score=score)
        return (*r, binding.balance_loss_backward(one, l, r[1], r[3], k, offsets=off, score=score))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for src in (near, far, near):
        l.copy_(src)
        g.replay()
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert all(torch.isfinite(x.float()).all() for x in got) and (got[4][-3:] == 0).all()
