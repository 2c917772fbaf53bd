"""Block-scaled FP8 product (moe_gemm_fp8) against the float64 definition.

Most tests are exact: codes that are small integers and scales that are small integers (fp32) or powers of two
(UE8M0), so that every partial sum in any order is a multiple of the unit below 2^24 units and fp32 makes no
rounding; an fp32 output then equals the definition, a bf16 output its one rounding.  With scales of 1 to 5
on both sides (25), codes to 8 (64) and K <= 1100 the sums stay below 1.8e6 < 2^24; with powers of two from
2^-1 to 2 the unit is 2^-2 and the sums below 1100 * 64 * 4 * 4 = 1.2e6 units.

With ordinary values the tolerance is K 1.1 2^-23 of the sum of magnitudes: an MMA adds 32 products and the
accumulator, each truncated to 24 bits or more below the largest of them (33 * 2^-23 of it at most), K / 32 times;
the scaling and adding of K / 128 block sums in fp32 is 3 * 2^-24 each, within the 1.1; bf16 adds 2^-8 of
the result."""
import numpy as np
import pytest
import torch

from fp8_fp4_moe_b200 import binding
from oracle import training as O

pytestmark = pytest.mark.gpu
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _codes(rng, R, K, fmt, pitch=None):
    """Small integers as FP8 codes, row pitch a multiple of 16 (the padding holds NaN codes)."""
    v = rng.integers(-8, 9, (R, K)).astype(np.float64) if fmt == "e4m3" else rng.choice([-8, -6, -4, -2, -1, 0, 1, 2, 3, 5], (R, K)).astype(np.float64)
    pitch = -(-K // 16) * 16 if pitch is None else pitch
    full = torch.full((R, pitch), 0x7F, dtype=torch.uint8, device="cuda")
    full[:, :K] = torch.from_numpy(O.encode_fp8(v, fmt)).cuda()
    return v, full.view(FP8[fmt])[:, :K]


def _scales(rng, R, K, per, kind, order="rows"):
    n = R if per == "row" else O.blocks(R)
    if kind == "ue8m0":
        c = rng.integers(126, 129, (n, O.blocks(K))).astype(np.uint8)
        s = np.exp2(c.astype(np.float64) - 127)
        t = torch.from_numpy(c).cuda()
    else:
        s = rng.integers(1, 6, (n, O.blocks(K))).astype(np.float64)
        t = torch.from_numpy(s).float().cuda()
    return s, (t.t().contiguous().t() if order == "rows" else t.contiguous())


def _case(seed, M, N, K, kind, a_per="row", b_per="tile", fa="e4m3", fb="e4m3", order="rows"):
    rng = np.random.default_rng(seed)
    a, A = _codes(rng, M, K, fa)
    b, B = _codes(rng, N, K, fb)
    sa, As = _scales(rng, M, K, a_per, kind, order)
    sb, Bs = _scales(rng, N, K, b_per, kind, order)
    return O.gemm(a, sa, b, sb)[0], A, As, B, Bs


def _equal(out, ws, ref):
    torch.cuda.synchronize()
    assert ws[:16].view(torch.int32)[0].item() == 0
    want = torch.from_numpy(ref)
    want = want.to(torch.bfloat16) if out.dtype == torch.bfloat16 else want.float()
    got = out.cpu()
    bad = (got != want).nonzero()
    assert bad.numel() == 0, (bad.shape[0], bad[:5].tolist(), got[tuple(bad[0])].item(), want[tuple(bad[0])].item())


SIZES = [(1, 1, 1), (1, 128, 128), (1, 1000, 1024), (3, 17, 130), (16, 256, 512), (17, 300, 1000), (31, 129, 640), (33, 640, 48),
         (64, 512, 1024), (65, 128, 257), (100, 1100, 900), (128, 384, 1024), (129, 256, 384), (130, 1, 200), (200, 130, 1100),
         (300, 512, 128), (333, 777, 555), (513, 1024, 300), (1000, 60, 1024), (257, 2049, 1000)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind", ["fp32", "ue8m0"])
@pytest.mark.parametrize("b_per", ["row", "tile"])
def test_exact(cuda_lib, M, N, K, kind, b_per):
    ref, *op = _case(M + N + K, M, N, K, kind, b_per=b_per)
    _equal(*binding.gemm_fp8(*op, out_dtype=torch.float32), ref)
    _equal(*binding.gemm_fp8(*op), ref)


@pytest.mark.parametrize("M,N,K", [(5, 200, 300), (70, 256, 1024), (200, 300, 260)])
@pytest.mark.parametrize("kind", ["fp32", "ue8m0"])
@pytest.mark.parametrize("a_per", ["row", "tile"])
@pytest.mark.parametrize("fa,fb", [("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")])
def test_exact_formats_and_scale_blocks(cuda_lib, M, N, K, kind, a_per, fa, fb):
    ref, *op = _case(M * N + K, M, N, K, kind, a_per=a_per, fa=fa, fb=fb, order="columns")
    _equal(*binding.gemm_fp8(*op, out_dtype=torch.float32), ref)


@pytest.mark.parametrize("M,N,K", [(1, 300, 3584), (20, 128, 3600), (64, 512, 7168), (128, 200, 2049), (300, 256, 1537)])
@pytest.mark.parametrize("kind", ["fp32", "ue8m0"])
@pytest.mark.parametrize("order", ["rows", "columns"])
def test_exact_long_k(cuda_lib, M, N, K, kind, order):
    # K loops split over CTAs at block counts that are and are not multiples of four, scales of a row or of a column
    # next to each other; codes of -1, 0 and 1, so that the sums stay below 7168 * 25 (fp32) and 7168 * 16 units
    rng = np.random.default_rng(K)
    a, A = _codes(rng, M, K, "e4m3")
    b, B = _codes(rng, N, K, "e4m3")
    for v, t in ((a, A), (b, B)):
        np.sign(v, out=v)
        t.view(torch.uint8).copy_(torch.from_numpy(O.encode_fp8(v, "e4m3")))
    sa, As = _scales(rng, M, K, "row", kind, order)
    sb, Bs = _scales(rng, N, K, "tile", kind, order)
    _equal(*binding.gemm_fp8(A, As, B, Bs, out_dtype=torch.float32), O.gemm(a, sa, b, sb)[0])


@pytest.mark.parametrize("M,N,K", [(128, 30000, 256), (70, 9000, 400), (16, 40000, 130), (129, 128, 4096), (140, 20000, 128),
                                   (2000, 64, 512), (4097, 1, 256), (1, 40001, 128), (600, 5000, 256)])
@pytest.mark.parametrize("kind", ["fp32", "ue8m0"])
def test_exact_cuts(cuda_lib, M, N, K, kind):
    # sizes at which the tiles are cut in each of the ways: column tiles of 16 to 256, one and two CTAs, split K loops
    rng = np.random.default_rng(M + N)
    a, A = _codes(rng, M, K, "e4m3")
    b, B = _codes(rng, N, K, "e4m3")
    if K > 1100:                                         # codes of -1, 0 and 1
        for v, t in ((a, A), (b, B)):
            np.sign(v, out=v)
            t.view(torch.uint8).copy_(torch.from_numpy(O.encode_fp8(v, "e4m3")))
    for per in ("row", "tile"):
        sa, As = _scales(rng, M, K, "row", kind)
        sb, Bs = _scales(rng, N, K, per, kind)
        x = torch.from_numpy(O.dequant(a, sa)).cuda()
        y = torch.from_numpy(O.dequant(b, sb)).cuda()
        _equal(*binding.gemm_fp8(A, As, B, Bs, out_dtype=torch.float32), (x @ y.T).cpu().numpy())


@pytest.mark.parametrize("seed", range(24))
def test_exact_random_sizes(cuda_lib, seed):
    rng = np.random.default_rng(1000 + seed)
    M, N, K = (int(np.exp(rng.uniform(0, np.log(top)))) for top in (1500, 3000, 1100))
    kind, order = rng.choice(["fp32", "ue8m0"]), rng.choice(["rows", "columns"])
    a_per, b_per = rng.choice(["row", "tile"]), rng.choice(["row", "tile"])
    ref, *op = _case(seed, M, N, K, kind, a_per=a_per, b_per=b_per, fa=rng.choice(["e4m3", "e5m2"]),
                     fb=rng.choice(["e4m3", "e5m2"]), order=order)
    dtype = torch.float32 if rng.random() < 0.5 else torch.bfloat16
    _equal(*binding.gemm_fp8(*op, out_dtype=dtype), ref)


@pytest.mark.parametrize("M,N,K", [(9, 200, 300), (129, 260, 1024), (700, 513, 128)])
@pytest.mark.parametrize("kind", ["fp32", "ue8m0"])
def test_accumulate_strided_and_unaligned_outputs(cuda_lib, M, N, K, kind):
    ref, *op = _case(M + 2 * N, M, N, K, kind)
    # pitches and starts that allow 16-byte stores and that do not; what lies around stays as it was
    for pitch, first in ((N + 16 - N % 4, 4), (N + 3, 1)):
        for dtype, acc in ((torch.float32, True), (torch.float32, False), (torch.bfloat16, False)):
            big = torch.full((M + 2, pitch + 4), 3.0, dtype=dtype, device="cuda")
            out = big[1:M + 1, first:first + N]
            got, ws = binding.gemm_fp8(*op, out=out, accumulate=acc)
            assert got is out
            _equal(out, ws, ref + 3.0 if acc else ref)
            big[1:M + 1, first:first + N] = 3.0
            assert (big == 3).all()


def test_many_tiles_and_bands(cuda_lib):
    # more tiles than SMs, several bands of row tiles, ragged last tiles
    for kind in ("fp32", "ue8m0"):
        ref, *op = _case(1, 2500, 3001, 260, kind)
        _equal(*binding.gemm_fp8(*op, out_dtype=torch.float32), ref)
        ref, *op = _case(2, 2500, 3001, 100, kind, b_per="row")
        _equal(*binding.gemm_fp8(*op), ref)


@pytest.mark.parametrize("M,N,K", [(1, 512, 2048), (40, 256, 7168), (300, 300, 1000), (256, 512, 4096)])
@pytest.mark.parametrize("kind", ["fp32", "ue8m0"])
@pytest.mark.parametrize("fa", ["e4m3", "e5m2"])
def test_ordinary_values(cuda_lib, M, N, K, kind, fa):
    g = torch.Generator().manual_seed(M + K)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    w = torch.randn(N, K, generator=g)
    sd = torch.uint8 if kind == "ue8m0" else torch.float32
    A, As, _, _ = binding.quant_fp8(x.cuda(), dtype=FP8[fa], scale_dtype=sd)
    B, Bs, _, _ = binding.quant_fp8(w.cuda(), block="tile", scale_dtype=sd)
    if kind == "fp32":                                   # scales of a checkpoint need not be powers of two
        As, Bs = As * 1.37, Bs * 0.71
    num = lambda s: np.exp2(s.cpu().double().numpy() - 127) if s.dtype == torch.uint8 else s.cpu().double().numpy()  # noqa: E731
    a = O.decode_fp8(A.contiguous().view(torch.uint8).cpu().numpy(), fa)
    b = O.decode_fp8(B.contiguous().view(torch.uint8).cpu().numpy(), "e4m3")
    ref, mag = O.gemm(a, num(As), b, num(Bs))
    for dtype in (torch.float32, torch.bfloat16):
        out, ws = binding.gemm_fp8(A, As, B, Bs, out_dtype=dtype)
        torch.cuda.synchronize()
        assert ws[:4].view(torch.int32).item() == 0
        err = np.abs(out.double().cpu().numpy() - ref)
        tol = K * 1.1 * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0)
        assert (err <= tol).all(), (err / tol).max()


def test_nan_and_extreme_scales_stay_in_their_rows(cuda_lib):
    for kind in ("fp32", "ue8m0"):
        ref, A, As, B, Bs = _case(3, 150, 200, 300, kind, b_per="row")
        A.view(torch.uint8)[7, 250] = 0x7F               # a NaN code
        As[9, 1] = 255 if kind == "ue8m0" else float("nan")
        Bs[11, 0] = 255 if kind == "ue8m0" else float("nan")
        out, _ = binding.gemm_fp8(A, As, B, Bs, out_dtype=torch.float32)
        got = out.cpu().numpy()
        bad = np.zeros(got.shape, bool)
        bad[7], bad[9], bad[:, 11] = True, True, True
        assert np.isnan(got[bad]).all()
        np.testing.assert_array_equal(got[~bad], ref[~bad].astype(np.float32))


def test_broadcast_scales_and_plain_bytes(cuda_lib):
    rng = np.random.default_rng(4)
    a, A = _codes(rng, 140, 260, "e4m3")
    b, B = _codes(rng, 150, 260, "e4m3")
    one = torch.full((1, 1), 2.0, device="cuda")
    out = binding.gemm_fp8(A.view(torch.uint8), one.expand(140, 3), B.view(torch.uint8), one.expand(2, 3), out_dtype=torch.float32)
    _equal(*out, 4 * (a @ b.T))


def test_empty(cuda_lib):
    f8 = FP8["e4m3"]
    z = lambda *s: torch.zeros(*s, device="cuda")        # noqa: E731
    for M, N, K in ((0, 8, 256), (8, 0, 256), (5, 9, 0), (0, 0, 0)):
        A, B, kb = z(M, K).to(f8), z(N, K).to(f8), -(-K // 128)
        out, ws = binding.gemm_fp8(A, z(M, kb), B, z(N, kb))
        assert out.shape == (M, N) and (out == 0).all() and ws[:4].view(torch.int32).item() == 0
    big = torch.full((5, 12), 3.0, device="cuda")
    binding.gemm_fp8(z(5, 0).to(f8), z(5, 0), z(9, 0).to(f8), z(9, 0), out=big[:, :9], accumulate=True)
    assert (big == 3).all()
    binding.gemm_fp8(z(5, 0).to(f8), z(5, 0), z(9, 0).to(f8), z(9, 0), out=big[:, :9])
    assert (big[:, :9] == 0).all() and (big[:, 9:] == 3).all()


def test_two_streams_and_graphs(cuda_lib):
    cases = [_case(20 + i, 60 + 90 * i, 300, 1024, kind) for i, kind in enumerate(("fp32", "ue8m0", "fp32", "ue8m0"))]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [binding.gemm_fp8(*c[1:], out_dtype=torch.float32, stream=s) for _ in range(3) for c, s in zip(cases, streams)][-4:]
    torch.cuda.synchronize()
    for (out, ws), c in zip(outs, cases):
        _equal(out, ws, c[0])
    # a captured product follows its operands
    ref, A, As, B, Bs = _case(30, 200, 260, 512, "fp32")
    ref2, A2, As2, B2, Bs2 = _case(31, 200, 260, 512, "fp32")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    graphs = []
    for _ in range(2):                                   # two graphs may share a workspace when they run in turn
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, _ = binding.gemm_fp8(A, As, B, Bs, workspace=ws, out_dtype=torch.float32)
        graphs.append((g, out))
    for g, out in graphs:
        g.replay()
        _equal(out, ws, ref)
    for t, u in ((A, A2), (B, B2)):
        t.view(torch.uint8).copy_(u.view(torch.uint8))
    As.copy_(As2)
    Bs.copy_(Bs2)
    for g, out in graphs:
        g.replay()
        _equal(out, ws, ref2)


@pytest.mark.parametrize("T,H,N,scale_dtype", [(1, 256, 512, torch.float32), (77, 512, 384, torch.uint8), (1000, 640, 300, torch.float32)])
def test_training_step_of_a_linear_layer(cuda_lib, T, H, N, scale_dtype):
    """Forward, input gradient and weight gradient of y = x W^T from quantised operands, each against the
    float64 product of the values that its codes stand for; the weight gradient over two micro-batches."""
    g = torch.Generator().manual_seed(T)
    x, dy = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda(), torch.randn(T, N, generator=g).to(torch.bfloat16).cuda()
    w = torch.randn(N, H, generator=g).cuda()
    kw = dict(scale_dtype=scale_dtype)
    qx = binding.quant_fp8(x, cols=True, **kw)
    qw = binding.quant_fp8(w, block="tile", cols=True, **kw)
    qd = binding.quant_fp8(dy, cols=True, dtype=FP8["e5m2"], **kw)
    y, _ = binding.gemm_fp8(qx[0], qx[1], qw[0], qw[1])
    dx, _ = binding.gemm_fp8(qd[0], qd[1], qw[2], qw[3])
    dw = torch.zeros(N, H, device="cuda")
    for _ in range(2):
        binding.gemm_fp8(qd[2], qd[3], qx[2], qx[3], out=dw, accumulate=True)

    def value(q, s):
        fmt = "e5m2" if q.dtype == FP8["e5m2"] else "e4m3"
        s = np.exp2(s.cpu().double().numpy() - 127) if s.dtype == torch.uint8 else s.cpu().double().numpy()
        return O.dequant(O.decode_fp8(q.contiguous().view(torch.uint8).cpu().numpy(), fmt), s)

    for got, (a, sa), (b, sb), times in ((y, qx[:2], qw[:2], 1), (dx, qd[:2], qw[2:], 1), (dw, qd[2:], qx[2:], 2)):
        a, b = value(a, sa), value(b, sb)
        ref, mag, K = times * (a @ b.T), times * (np.abs(a) @ np.abs(b).T), a.shape[1]
        tol = (K * 1.1 + 2) * 2.0 ** -23 * mag + (2.0 ** -8 * np.abs(ref) if got.dtype == torch.bfloat16 else 0)
        assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all()
    # and near the product of the unquantised values: each operand is off by at most half a step of its format, 2^-4
    # (E4M3) or 2^-3 (E5M2) of the element (codes below the format's normal range: of amax 2^-15 at most)
    xd, wd = x.double().cpu().numpy(), w.double().cpu().numpy()
    assert (np.abs(y.double().cpu().numpy() - xd @ wd.T) <= (2 * 2.0 ** -4 + 2.0 ** -7) * 1.01 * (np.abs(xd) @ np.abs(wd).T) + 1e-2 * np.sqrt(H)).all()


@pytest.mark.parametrize("kind", ["fp32", "ue8m0"])
def test_offsets_beyond_32_bits(cuda_lib, kind):
    """An output of more than 2^31 elements, and operand rows more than 2^31 bytes apart."""
    M, N, K = 66000, 32776, 130
    st = torch.float32 if kind == "fp32" else torch.uint8
    x = torch.randn(M, K, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(N, K, device="cuda", dtype=torch.bfloat16)
    A, As, _, _ = binding.quant_fp8(x, scale_dtype=st)
    B, Bs, _, _ = binding.quant_fp8(w, block="tile", scale_dtype=st)
    out, _ = binding.gemm_fp8(A, As, B, Bs)
    tail, _ = binding.gemm_fp8(A[-200:], As[-200:], B, Bs)
    assert torch.equal(out[-200:], tail)
    head, _ = binding.gemm_fp8(A[:200], As[:200], B, Bs)
    assert torch.equal(out[:200], head)
    del out
    wide = torch.empty(M, 32784, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, 16:16 + K]
    wide.copy_(A)
    narrow = B[:300]
    Bs300 = Bs[:3]
    a, _ = binding.gemm_fp8(wide, As, narrow, Bs300)
    b, _ = binding.gemm_fp8(A, As, narrow, Bs300)
    assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["fp32", "ue8m0"])
def test_product_with_itself(cuda_lib, kind):
    rng = np.random.default_rng(40)
    a, A = _codes(rng, 300, 400, "e4m3")
    s, As = _scales(rng, 300, 400, "row", kind)
    out, ws = binding.gemm_fp8(A, As, A, As, out_dtype=torch.float32)
    _equal(out, ws, O.gemm(a, s, a, s)[0])


@pytest.mark.parametrize("scale_dtype", [torch.float32, torch.uint8])
@pytest.mark.parametrize("M", [1, 100, 700])
def test_captured_layer_step_follows_its_inputs(cuda_lib, M, scale_dtype):
    """Copies, memsets, two branches that join, and calls that follow one another without a gap, as one graph: replayed on
    new inputs it gives what the calls give one by one."""
    N, K = 520, 384
    src = torch.empty(M, K, device="cuda", dtype=torch.bfloat16)
    src2 = torch.empty(N, K, device="cuda", dtype=torch.bfloat16)
    x, w = torch.empty_like(src), torch.empty_like(src2)
    acc = torch.empty(M, N, device="cuda")
    side = torch.cuda.Stream()

    def step():
        main = torch.cuda.current_stream()
        x.copy_(src)
        acc.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            w.copy_(src2)
            B, Bs, _, _ = binding.quant_fp8(w, block="tile", scale_dtype=scale_dtype)
        A, As, _, _ = binding.quant_fp8(x, scale_dtype=scale_dtype)
        main.wait_stream(side)
        y, ws = binding.gemm_fp8(A, As, B, Bs)
        binding.gemm_fp8(A, As, B, Bs, out=acc, accumulate=True, workspace=ws)
        binding.gemm_fp8(A, As, B, Bs, out=acc, accumulate=True, workspace=ws)
        q, s, _, _ = binding.quant_fp8(y, scale_dtype=scale_dtype)
        z, _ = binding.gemm_fp8(q, s, q, s, workspace=ws, out_dtype=torch.float32)
        return y, acc.clone(), z, ws

    src.normal_(), src2.normal_()
    torch.cuda.synchronize()
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for _ in range(5):
        src.normal_(), src2.normal_()
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        have = [t.clone() for t in got]
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(have[:3], want[:3]):
            assert torch.equal(a, b)
        assert have[3][:16].view(torch.int32)[0].item() == 0


@pytest.mark.parametrize("M,N,K", [(300, 5000, 2000), (520, 7001, 1300), (300, 5888, 2048)])
@pytest.mark.parametrize("b_per", ["row", "tile"])
def test_exact_pair_tiles_of_224_columns(cuda_lib, M, N, K, b_per):
    """One wave of CTA pairs (column scales: 224 columns, 112 to each half).  Sums stay below 25 * 64 * 2048 = 3.3e6 <
    2^24 units, also with 7000 added."""
    ref, A, As, B, Bs = _case(50, M, N, K, "fp32", b_per=b_per)
    out, ws = binding.gemm_fp8(A, As, B, Bs)
    _equal(out, ws, ref)
    acc = torch.full((M, N), 7000.0, device="cuda")
    binding.gemm_fp8(A, As, B, Bs, out=acc, accumulate=True, workspace=ws)
    _equal(acc, ws, ref + 7000)
