"""Balance loss and its gradient against the float64 definition.

Tolerances (u = 2^-24, fp32's unit roundoff).  A score is exp(l - m) / sum: the rounding of l - m (|l - m| <= 32
here, so 32 u relative to the exponential), expf (2 ulp = 4 u), the row sum over E <= 1024 terms of one sign in
32 lanes (E / 32 + 5 additions <= 37 u), a reciprocal and a product (2 u): at most 32 + 4 twice (term and sum) +
37 + 2 < 112 u.  The sigmoid's has expf, an addition and a division (6 u) in place of the difference.  Scores are then
added over at most T tokens, all of one sign: T u.  probs: (T + 112 + 2) u relative.  The loss adds its terms
in 64 bits.  The gradient g p (c - mean) has p (112 u) and mean (112 u + E / 32 + 5 additions, 37 u) and the
rounding of c (u), g (8 u) and three products: below 300 u of g p (c + mean); 1 - sigma adds 8 u of 1 (not of itself).
bf16 adds its half ulp, 2^-8."""
import numpy as np
import pytest
import torch

from fp8_fp4_moe_b200 import binding
from oracle import training as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _inputs(seed, T, E, k, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    l = (torch.randn(T, E, generator=g) * 2 + torch.randn(1, E, generator=g)).to(dtype)
    ids = torch.topk(l.float(), k, dim=1).indices.to(torch.int32)
    return l, ids


def _cut(seed, T, S):
    r = np.random.default_rng(seed)
    return torch.tensor(np.sort(r.integers(0, T + 1, S + 1)), dtype=torch.int32)


def _check(l, ids, offsets=None, mask=None, score="softmax", coef=0.01, grad_loss=1.5, logits=None):
    T, E = l.shape
    k = ids.shape[1]
    dl = l.cuda() if logits is None else logits
    do, dm = (None if v is None else v.cuda() for v in (offsets, mask))
    args = dict(coef=coef, offsets=do, mask=dm, score=score)
    loss, counts, probs, tokens = binding.balance_loss(dl, ids.cuda(), **args)
    grad = binding.balance_loss_backward(torch.tensor(grad_loss, device="cuda"), dl, counts, tokens, k, **args)
    v, o, m = l.double().numpy(), None if offsets is None else offsets.numpy(), None if mask is None else mask.numpy()
    ref_loss, ref_c, ref_p, ref_n, _ = O.balance_loss(v, ids.numpy(), coef, o, m, score)
    ref_g, mag = O.balance_grad(grad_loss, v, ids.numpy(), coef, o, m, score)
    np.testing.assert_array_equal(counts.cpu().numpy(), ref_c)
    np.testing.assert_array_equal(tokens.cpu().numpy(), ref_n)
    rel = (T + 114) * U
    assert (np.abs(probs.cpu().numpy() - ref_p) <= rel * ref_p + 1e-37).all()
    assert abs(loss.item() - ref_loss) <= (rel + 2 * U) * abs(ref_loss)
    got = grad.double().cpu().numpy()
    tol = 300 * U * mag + 1e-37
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            f = np.exp(-np.maximum(v, 0) - np.log1p(np.exp(-np.abs(v))))
        tol = tol + 8 * U * mag / np.maximum(f, 1e-30)
    if l.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(ref_g)
    assert grad.dtype == l.dtype
    assert (np.abs(got - ref_g) <= tol).all(), np.max(np.abs(got - ref_g) / tol)
    return loss, counts, probs, tokens, grad


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 3, 3), (64, 8, 2), (33, 31, 4), (100, 33, 16), (512, 256, 8),
                                   (301, 257, 8), (40, 1000, 8), (77, 1024, 5), (3000, 64, 6)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_whole_batch(cuda_lib, T, E, k, score, dtype):
    l, ids = _inputs(T + E, T, E, k, dtype)
    _check(l, ids, score=score)


@pytest.mark.parametrize("T,E,S", [(1, 8, 3), (50, 16, 7), (700, 256, 5), (513, 100, 200), (2500, 8, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("masked", [0.0, 0.4, 1.0])
def test_packed_sequences_and_masks(cuda_lib, T, E, S, score, masked):
    l, ids = _inputs(T + S, T, E, 2)
    mask = torch.rand(T, generator=torch.Generator().manual_seed(S)) >= masked if masked else None
    _check(l, ids, offsets=_cut(T + S, T, S), mask=mask, score=score)
    _check(l, ids, mask=mask, score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(cuda_lib, score):
    l, ids = _inputs(5, 40, 48, 4)
    low = torch.finfo(torch.float32).min
    l[0] = float("-inf")                                  # nothing left
    l[1, 1:] = float("-inf")
    l[2, ::2] = low                                       # the type's lowest value as a mask
    l[3] = low
    l[4] = 0
    l[5] = -2000.0                                        # every sigmoid underflows
    l[6, 3] = 20.0
    ids[7] = torch.tensor([-1, 48, 5, 5], dtype=torch.int32)   # not experts; one expert twice
    loss, counts, probs, tokens, grad = _check(l, ids, score=score)
    assert torch.isfinite(grad).all() and torch.isfinite(probs).all()
    assert (grad[0] == 0).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_equal_counts_have_no_gradient(cuda_lib, score):
    # every token takes every expert: the loss is coef whatever the scores
    l, _ = _inputs(11, 50, 8, 8)
    ids = torch.arange(8, dtype=torch.int32).expand(50, 8).contiguous()
    loss, counts, probs, tokens = binding.balance_loss(l.cuda(), ids.cuda(), coef=0.5, score=score)
    grad = binding.balance_loss_backward(torch.ones((), device="cuda"), l.cuda(), counts, tokens, 8, coef=0.5, score=score)
    assert (grad == 0).all() and abs(loss.item() - 0.5) <= 0.5 * (50 + 114) * U


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [8, 64, 600])
def test_gradient_beside_a_popular_expert_of_low_score(cuda_lib, score, E):
    # all choose expert 0, whose score is small: the others' gradient, p (0 - mean) with a mean near 0, keeps its digits
    l, _ = _inputs(12, 300, E, 1)
    l[:, 0] -= 20
    _check(l, torch.zeros(300, 1, dtype=torch.int32), score=score)
    off = torch.tensor([0, 7, 7, 130, 301 - 1], dtype=torch.int32)
    _check(l, torch.zeros(300, 1, dtype=torch.int32), offsets=off, score=score)


def test_infinite_logits(cuda_lib):
    # sigmoid(inf) is 1; a softmax with an infinity is undefined, in its row alone
    l, ids = _inputs(13, 30, 16, 2)
    l[4, 5] = float("inf")
    args = dict(coef=0.01, score="sigmoid")
    loss, counts, probs, tokens = binding.balance_loss(l.cuda(), ids.cuda(), **args)
    grad = binding.balance_loss_backward(torch.ones((), device="cuda"), l.cuda(), counts, tokens, 2, **args)
    v, n = l.double().numpy(), ids.numpy()
    p = O.scores(v, "sigmoid")
    c = O.balance_loss(v, n, 0.01, score="sigmoid")[1]
    whole = 0.01 * 16 / 2 / 30 / 30 * p * (c + (p * c).sum(1, keepdims=True))   # the magnitudes without 1 - sigma
    ref, mag = O.balance_grad(1.0, v, n, 0.01, score="sigmoid")
    assert ref[4, 5] == 0 and (np.abs(grad.cpu().numpy() - ref) <= U * (300 * mag + 8 * whole)).all()
    assert abs(loss.item() - O.balance_loss(v, n, 0.01, score="sigmoid")[0]) <= (30 + 116) * U * loss.item()
    loss, counts, probs, tokens = binding.balance_loss(l.cuda(), ids.cuda())
    grad = binding.balance_loss_backward(torch.ones((), device="cuda"), l.cuda(), counts, tokens, 2)
    assert torch.isnan(loss) and torch.isnan(grad[4]).any()
    assert torch.isfinite(grad[:4]).all() and torch.isfinite(grad[5:]).all()


def test_what_a_mask_hides_is_not_read(cuda_lib):
    l, ids = _inputs(6, 100, 64, 3)
    mask = torch.ones(100, dtype=torch.bool)
    mask[10:20] = False
    off = torch.tensor([5, 50, 80], dtype=torch.int32)
    want = _check(l, ids, offsets=off, mask=mask)
    bad = l.clone()
    bad[10:20] = float("nan")
    bad[:5] = float("inf")
    bad[80:] = float("nan")
    args = dict(coef=0.01, offsets=off.cuda(), mask=mask.cuda())
    got = binding.balance_loss(bad.cuda(), ids.cuda(), **args)
    grad = binding.balance_loss_backward(torch.tensor(1.5, device="cuda"), bad.cuda(), got[1], got[3], 3, **args)
    for a, b in zip(want, (*got, grad)):
        assert torch.equal(a, b)
    assert (grad[10:20] == 0).all() and (grad[:5] == 0).all() and (grad[80:] == 0).all()
    # a NaN that does count is seen
    bad = l.clone()
    bad[30, 7] = float("nan")
    got = binding.balance_loss(bad.cuda(), ids.cuda(), **args)
    assert torch.isnan(got[0]) and torch.isnan(got[2][0]).any() and torch.isfinite(got[2][1]).all()


def test_strides_accumulate_and_in_place(cuda_lib):
    l, ids = _inputs(7, 90, 60, 2)
    wide = torch.full((90, 71), float("nan"), device="cuda")
    wide[:, 3:63] = l.cuda()
    want = _check(l, ids)
    _check(l, ids, logits=wide[:, 3:63])
    g = torch.tensor(1.5, device="cuda")
    out = torch.zeros(90, 80, device="cuda")
    out += 2.0
    binding.balance_loss_backward(g, l.cuda(), want[1], want[3], 2, coef=0.01, out=out[:, 1:61], accumulate=True)
    assert torch.equal(out[:, 1:61], want[4] + 2.0) and (out[:, :1] == 2).all() and (out[:, 61:] == 2).all()
    buf = l.cuda()
    got = binding.balance_loss_backward(g, buf, want[1], want[3], 2, coef=0.01, out=buf)
    assert got is buf and torch.equal(buf, want[4])
    # tokens that do not count stay as they were
    mask = torch.ones(90, dtype=torch.bool, device="cuda")
    mask[4] = False
    out = torch.full((90, 60), 3.0, device="cuda")
    c = binding.balance_loss(l.cuda(), ids.cuda(), mask=mask)
    binding.balance_loss_backward(g, l.cuda(), c[1], c[3], 2, mask=mask, out=out, accumulate=True)
    assert (out[4] == 3).all() and not (out[5] == 3).all()


def test_no_tokens(cuda_lib):
    l = torch.zeros(0, 16, device="cuda")
    ids = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    loss, counts, probs, tokens = binding.balance_loss(l, ids)
    assert loss.item() == 0 and (counts == 0).all() and (probs == 0).all() and (tokens == 0).all()
    assert binding.balance_loss_backward(torch.ones((), device="cuda"), l, counts, tokens, 2).shape == (0, 16)


def test_runs_repeat_on_another_stream_and_in_a_graph(cuda_lib):
    l, ids = _inputs(8, 2000, 256, 8)
    dl, di, g = l.cuda(), ids.cuda(), torch.tensor(0.7, device="cuda")

    def step(stream=None):
        r = binding.balance_loss(dl, di, stream=stream)
        return (*r, binding.balance_loss_backward(g, dl, r[1], r[3], 8, stream=stream))

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    l2, ids2 = _inputs(9, 2000, 256, 8)
    dl.copy_(l2)
    di.copy_(ids2)
    graph.replay()
    want = step()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_offsets_that_do_not_ascend_stay_in_bounds(cuda_lib):
    # values are unspecified, but nothing outside the arrays is touched
    l, ids = _inputs(10, 64, 32, 2)
    pad = torch.full((66, 32), 7.0, device="cuda")
    off = torch.tensor([40, -5, 1000, 3, 64], dtype=torch.int32, device="cuda")
    loss, counts, probs, tokens = binding.balance_loss(l.cuda(), ids.cuda(), offsets=off)
    binding.balance_loss_backward(torch.ones((), device="cuda"), l.cuda(), counts, tokens, 2, offsets=off, out=pad[1:65])
    torch.cuda.synchronize()
    assert (pad[0] == 7).all() and (pad[65] == 7).all()


def test_offsets_beyond_32_bits(cuda_lib):
    """More than 2^31 logits: the last sequence's results are those of its tokens alone."""
    T, E, k, tail = (1 << 23) + 77, 257, 2, 900
    l = torch.empty(T, E, dtype=torch.bfloat16, device="cuda")
    l.uniform_(-3, 3)
    ids = torch.randint(0, E, (T, k), dtype=torch.int32, device="cuda")
    off = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    one = torch.ones((), device="cuda")
    loss, counts, probs, tokens = binding.balance_loss(l, ids, offsets=off)
    grad = binding.balance_loss_backward(one, l, counts, tokens, k, offsets=off)
    _, c, p, n, g = _check(l[-tail:].cpu(), ids[-tail:].cpu())
    g = binding.balance_loss_backward(one, l[-tail:], c, n, k, coef=0.5)       # half the loss: one of two sequences
    assert torch.equal(counts[1], c[0]) and tokens.tolist() == [T - tail, tail]
    assert (probs[1] - p[0]).abs().max() <= 2 * (tail + 114) * U * p.max()
    assert (grad[-tail:].float() - g.float()).abs().max() <= 2.0 ** -7 * g.float().abs().max()
    assert int(counts[0].sum()) == (T - tail) * k
