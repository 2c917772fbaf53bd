"""Block scales at the ends of their type's range.

Codes are small whole numbers and scales powers of two, so every term is exact where fp32 holds it.  Codes are
not negative and a row (column) has one scale of its own, or a block of zeros, in each K block, chosen so that a result's
terms have the same magnitude or are zero: sums are exact above 2^-126, below they are off by half a step of
2^-149 per term and addition at most, and results beyond fp32's range are infinite."""
import numpy as np
import pytest
import torch

from fp8_fp4_moe_b200 import binding
from oracle import training as O

pytestmark = pytest.mark.gpu
SIZES = [(1, 300, 520), (5, 200, 300), (20, 128, 640), (60, 300, 1024), (100, 260, 4096), (200, 300, 260), (300, 700, 384),
         (520, 5000, 384), (300, 5888, 640)]


def _operand(rng, R, K, exps, per, zero):
    """Codes in 0..8 as values and FP8; block scales 2^e (fp32); a block of zeros wherever `zero` says so."""
    n = R if per == "row" else O.blocks(R)
    v = rng.integers(0, 9, (R, K)).astype(np.float64)
    e = rng.choice(exps, n)[:, None].repeat(O.blocks(K), 1)
    if zero:                                       # zeros under a scale near the top, on every other block
        e[:, 1::2] = 126
        for b in range(1, O.blocks(K), 2):
            v[:, 128 * b:128 * (b + 1)] = 0
    q = torch.zeros(R, -(-K // 16) * 16, dtype=torch.uint8)
    q[:, :K] = torch.from_numpy(O.encode_fp8(v, "e4m3"))
    return v, e, q.cuda().view(torch.float8_e4m3fn)[:, :K]


def _compare(out, ws, ref, K):
    torch.cuda.synchronize()
    assert ws[:4].view(torch.int32).item() == 0
    got = out.double().cpu().numpy()
    with np.errstate(over="ignore"):
        want = ref.astype(np.float32).astype(np.float64)
    assert not np.isnan(got).any()
    ordinary = np.abs(ref) >= 2.0 ** -126
    np.testing.assert_array_equal(got[ordinary], want[ordinary])
    assert (np.abs(got - ref)[~ordinary] <= O.blocks(K) * 2.0 ** -149).all()


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("b_per", ["row", "tile"])
@pytest.mark.parametrize("zero", [False, True])
def test_fp32_scales_of_every_size(cuda_lib, M, N, K, b_per, zero):
    rng = np.random.default_rng(M + N)
    # products from 2^-240 to 2^240: both tiny, both huge, and opposite ends that meet in the middle
    ea, eb = [0, 3, 66, -66, 75, -75, 120, -120, -140], [0, 70, -73, -62, 100, -100, 119, -121]
    a, sa, A = _operand(rng, M, K, ea, "row", zero)
    b, sb, B = _operand(rng, N, K, eb, b_per, zero)
    x, y = O.dequant(a, np.exp2(sa.astype(float))), O.dequant(b, np.exp2(sb.astype(float)))
    ref = (torch.from_numpy(x).cuda() @ torch.from_numpy(y).cuda().T).cpu().numpy()
    f = lambda e: torch.from_numpy(np.exp2(e.astype(np.float64)).astype(np.float32)).cuda()   # noqa: E731
    out, ws = binding.gemm_fp8(A, f(sa), B, f(sb), out_dtype=torch.float32)
    _compare(out, ws, ref, K)


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("b_per", ["row", "tile"])
def test_ordinary_groups_between_extreme_ones(cuda_lib, M, N, K, b_per):
    # the scales of a row differ by K block: extreme ones cancel (2^e and 2^-e, e of the K block) next to ordinary ones
    rng = np.random.default_rng(M * 3 + N)
    a, sa, A = _operand(rng, M, K, [0, 1, 2], "row", False)
    b, sb, B = _operand(rng, N, K, [0, 1, 2], b_per, False)
    e = rng.choice([0, 0, 0, 80, -80, 118, -118], O.blocks(K))
    sa, sb = sa + e, sb - e
    x, y = O.dequant(a, np.exp2(sa.astype(float))), O.dequant(b, np.exp2(sb.astype(float)))
    f = lambda e: torch.from_numpy(np.exp2(e.astype(np.float64)).astype(np.float32)).cuda()   # noqa: E731
    out, ws = binding.gemm_fp8(A, f(sa), B, f(sb), out_dtype=torch.float32)
    ref = (torch.from_numpy(x).cuda() @ torch.from_numpy(y).cuda().T).cpu().numpy()
    _compare(out, ws, ref, K)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_e5m2_codes_at_their_ends(cuda_lib, M, N, K):
    # one code a row: block sums from 2^-32 to 2^31, under scales whose product alone is out of range
    rng = np.random.default_rng(M + K)
    A, B = torch.zeros(M, K), torch.zeros(N, K)
    A[torch.arange(M), 7] = torch.from_numpy(rng.choice([2.0 ** -16, 1.0, 2.0 ** 15], M)).float()
    B[:, 7] = torch.from_numpy(rng.choice([2.0 ** -16, 1.0, 2.0 ** 15], N)).float()
    ld = -(-K // 16) * 16
    dev = [torch.zeros(t.shape[0], ld, dtype=torch.float8_e5m2, device="cuda")[:, :K] for t in (A, B)]
    for d, t in zip(dev, (A, B)):
        d.copy_(t.cuda())
    ea, eb = rng.choice([0, 80, -80, 127, -126, -149], M), rng.choice([0, 70, -70, 126, -125], N)
    kb = O.blocks(K)
    f = lambda e: torch.from_numpy(np.exp2(e.astype(np.float64)).astype(np.float32)[:, None].repeat(kb, 1)).cuda()   # noqa: E731
    out, ws = binding.gemm_fp8(dev[0], f(ea), dev[1], f(eb), out_dtype=torch.float32)
    x, y = A.double().numpy() * np.exp2(ea.astype(float))[:, None], B.double().numpy() * np.exp2(eb.astype(float))[:, None]
    _compare(out, ws, x[:, 7:8] @ y[:, 7:8].T, K)


@pytest.mark.parametrize("M,N,K", SIZES)
def test_ue8m0_scales_that_cancel_and_zeros_under_large_ones(cuda_lib, M, N, K):
    rng = np.random.default_rng(M + 2 * K)
    a, sa, A = _operand(rng, M, K, [0], "row", True)
    b, sb, B = _operand(rng, N, K, [0], "row", True)
    e = rng.choice([0, 80, -80, 120, -120], O.blocks(K))
    e[1::2] = 0                                    # zeros there, under 2^126 on both sides
    sa, sb = sa + e, sb - e
    f = lambda e: torch.from_numpy((e + 127).astype(np.uint8)).cuda()   # noqa: E731
    out, ws = binding.gemm_fp8(A, f(sa), B, f(sb), out_dtype=torch.float32)
    x, y = O.dequant(a, np.exp2(sa.astype(float))), O.dequant(b, np.exp2(sb.astype(float)))
    _compare(out, ws, (torch.from_numpy(x).cuda() @ torch.from_numpy(y).cuda().T).cpu().numpy(), K)


@pytest.mark.parametrize("M,N,K", [(5, 200, 1300), (300, 700, 1300), (300, 5888, 640)])
@pytest.mark.parametrize("b_per", ["row", "tile"])
def test_captured_products_at_once_follow_their_scales(cuda_lib, M, N, K, b_per):
    # two streams in one graph, accumulated and not; scales that are ordinary in one replay and extreme in the next
    rng = np.random.default_rng(N)
    a, sa, A = _operand(rng, M, K, [0, 1], "row", False)
    b, sb, B = _operand(rng, N, K, [0, 1], b_per, False)
    f = lambda e: torch.from_numpy(np.exp2(e.astype(np.float64)).astype(np.float32)).cuda()   # noqa: E731
    As, Bs, acc = f(sa), f(sb), torch.zeros(M, N, device="cuda")
    As2, Bs2 = As.clone(), Bs.clone()
    side = torch.cuda.Stream()

    def step():
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            acc.zero_()
            binding.gemm_fp8(A, As2, B, Bs2, out=acc, accumulate=True)
        r = binding.gemm_fp8(A, As, B, Bs, out_dtype=torch.float32)
        torch.cuda.current_stream().wait_stream(side)
        return r

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, ws = step()
    kb = O.blocks(K)
    for shift in ([0] * kb, [100] * kb, rng.choice([0, 0, 90, -110], kb), [-120] * kb, [0] * kb):
        e, e2 = np.asarray(shift), -np.asarray(shift)[::-1]
        As.copy_(f(sa + e)), Bs.copy_(f(sb - e))
        As2.copy_(f(sa + e2)), Bs2.copy_(f(sb - e2))
        g.replay()
        x, y = O.dequant(a, np.exp2(sa.astype(float))), O.dequant(b, np.exp2(sb.astype(float)))
        ref = (torch.from_numpy(x).cuda() @ torch.from_numpy(y).cuda().T).cpu().numpy()
        _compare(out, ws, ref, K)
        _compare(acc, ws, ref, K)
