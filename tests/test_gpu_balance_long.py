"""Mean scores of one sequence that is millions of tokens long.

Every row holds the same logits, so each addition to a lane's running sum is rounded the same way and a
long chain of them drifts by up to its length times u = 2^-24.  A block adds at most 4096 tokens of up to 256 experts, 32 rows at
a time: 128 additions a lane, 2 over lanes and 7 over warps.  Over blocks the roundings are carried along (2 u, whatever their
number) and 32 sums added in pairs (5 u).  A score of 8 experts with logits as near as these is off by less than 4 + 4 u (difference
and exponential) twice, 3 additions, a reciprocal and a product, 21 u, the mean by 2 u: below 253 u in all with room
for the 112 u of a score of any row; the drift of one chain over 2^24 tokens is above it."""
import numpy as np
import pytest
import torch

from fp8_fp4_moe_b200 import binding
from oracle import training as O

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("T,E,offsets", [(1 << 24, 8, None), (1 << 26, 8, None), ((1 << 24) + 77, 8, [5, (1 << 24) - 100, (1 << 24) + 70])])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_mean_scores_do_not_drift(cuda_lib, T, E, offsets, score):
    row = torch.tensor([0.3, -0.7, 1.1, 0.05, -1.9, 0.64, -0.21, 0.9])
    l = row.to(torch.bfloat16).cuda().expand(T, E).contiguous()
    ids = torch.zeros(T, 1, dtype=torch.int32, device="cuda")
    off = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    loss, counts, probs, tokens = binding.balance_loss(l, ids, offsets=off, score=score)
    p = O.scores(l[:1].cpu().double().numpy(), score)
    assert (np.abs(probs.cpu().numpy() - p) <= 253 * U * p).all(), np.max(np.abs(probs.cpu().numpy() - p) / p) / U
    n = [T] if offsets is None else np.diff(offsets).tolist()
    assert tokens.tolist() == n and counts[:, 0].tolist() == n
    assert abs(loss.item() - E * p[0, 0]) <= 256 * U * E * p[0, 0]
