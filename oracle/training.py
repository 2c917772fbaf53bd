"""Float64 definitions of the FP8 training operators: block quantisation, the block-scaled product and the
router's balance loss with its gradient (numpy only, no code shared with the library)."""
from __future__ import annotations

import math

import numpy as np

# (mantissa bits, exponent bias, largest finite value)
FORMATS = {"e4m3": (3, 7, 448.0), "e5m2": (2, 15, 57344.0)}


def blocks(n: int) -> int:
    return -(-n // 128)


def decode_fp8(codes: np.ndarray, fmt: str) -> np.ndarray:
    """Values of FP8 codes (uint8); E4M3 has NaN at 0x7F / 0xFF, E5M2 infinities and NaNs as IEEE."""
    man, bias, _ = FORMATS[fmt]
    c = codes.astype(np.int64)
    e, m = (c & 0x7F) >> man, c & ((1 << man) - 1)
    mag = np.where(e == 0, m * 2.0 ** (1 - bias - man), (1 + m * 2.0 ** -man) * np.exp2((e - bias).astype(np.float64)))
    if fmt == "e4m3":
        mag = np.where((c & 0x7F) == 0x7F, np.nan, mag)
    else:
        mag = np.where(e == 31, np.where(m == 0, np.inf, np.nan), mag)
    return np.where(c & 0x80, -mag, mag)


def encode_fp8(v: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of float64 values, round to nearest even, saturating; NaN -> 0x7F."""
    man, bias, top = FORMATS[fmt]
    a = np.minimum(np.abs(np.where(np.isnan(v), 0.0, v)), top)
    e = np.maximum(np.frexp(a)[1] - 1, 1 - bias)
    steps = np.rint(np.ldexp(a, man - e)).astype(np.int64)      # in units of the value's last place
    code = np.where(steps >= (1 << man), ((e + bias) << man) + steps - (1 << man), steps)
    code = code | np.where(np.signbit(v), 0x80, 0)
    return np.where(np.isnan(v), 0x7F, code).astype(np.uint8)


def scale_exp(amax: float, top: float) -> int:
    """The smallest p >= -126 with amax <= top * 2^p; 0 for amax = 0; the largest fp32 scale's for inf."""
    if amax == 0:
        return 0
    if math.isinf(amax):
        return 128 - int(math.floor(math.log2(top)))
    p = -126
    m, e = math.frexp(amax)
    p = max(p, e - 1 - int(math.floor(math.log2(top))) - 1)
    while amax > math.ldexp(top, p):
        p += 1
    return p


def quant(x: np.ndarray, block: str, fmt: str):
    """x [M, K] float64 -> (codes uint8 [M, K], exponents int [M or ceil(M/128), ceil(K/128)])."""
    M, K = x.shape
    step = 1 if block == "row" else 128
    p = np.zeros((-(-M // step), blocks(K)), np.int64)
    q = np.zeros((M, K), np.uint8)
    for i in range(p.shape[0]):
        for j in range(p.shape[1]):
            part = x[i * step:(i + 1) * step, j * 128:(j + 1) * 128]
            a = np.abs(part)
            p[i, j] = scale_exp(float(np.max(np.where(np.isnan(a), 0, a))), FORMATS[fmt][2])
            q[i * step:(i + 1) * step, j * 128:(j + 1) * 128] = encode_fp8(np.ldexp(part, -int(p[i, j])), fmt)
    return q, p


def dequant(values: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """values [R, K] times their block scales ([R or ceil(R/128), ceil(K/128)])."""
    R, K = values.shape
    if scales.shape[0] != R:
        scales = np.repeat(scales, 128, axis=0)[:R]
    return values * np.repeat(scales, 128, axis=1)[:, :K]


def gemm(a, sa, b, sb):
    """(sum of products, sum of their magnitudes), both [M, N]."""
    x, y = dequant(a, sa), dequant(b, sb)
    return x @ y.T, np.abs(x) @ np.abs(y).T


def scores(l: np.ndarray, score: str) -> np.ndarray:
    """p [T, E]; a row of -inf has zero scores."""
    z = l if score == "softmax" else np.minimum(l, 0) - np.log1p(np.exp(-np.abs(l)))   # log sigma
    with np.errstate(invalid="ignore"):
        w = np.where(np.isneginf(z), 0.0, np.exp(z - z.max(1, keepdims=True)))
    s = w.sum(1, keepdims=True)
    return w / np.where(s == 0, 1, s)


def balance_loss(l, ids, coef=1.0, offsets=None, mask=None, score="softmax"):
    """(loss, counts [S, E], probs [S, E], tokens [S], spans): spans[s] = the token indices that count."""
    T, E = l.shape
    k = ids.shape[1]
    ends = [0, T] if offsets is None else [int(v) for v in offsets]
    S = len(ends) - 1
    spans = [[t for t in range(ends[s], ends[s + 1]) if mask is None or mask[t]] for s in range(S)]
    counts, probs = np.zeros((S, E), np.int64), np.zeros((S, E))
    for s, span in enumerate(spans):
        for t in span:
            for e in ids[t]:
                if 0 <= e < E:
                    counts[s, e] += 1
        if span:
            probs[s] = scores(l[span], score).mean(0)
    tokens = np.array([len(v) for v in spans])
    live = int((tokens > 0).sum())
    loss = sum(E / (k * n) * float((counts[s] * probs[s]).sum()) for s, n in enumerate(tokens) if n > 0)
    return (coef * loss / live if live else 0.0), counts, probs, tokens, spans


def balance_grad(grad_loss, l, ids, coef=1.0, offsets=None, mask=None, score="softmax"):
    """(gradient of grad_loss * loss by the logits, the magnitudes its difference is taken of)."""
    _, counts, _, tokens, spans = balance_loss(l, ids, coef, offsets, mask, score)
    E, k, live = l.shape[1], ids.shape[1], max(1, int((tokens > 0).sum()))
    grad, mag = np.zeros(l.shape), np.zeros(l.shape)
    for s, span in enumerate(spans):
        if not span:
            continue
        p = scores(l[span], score)
        g = grad_loss * coef / live * E / (k * tokens[s]) / tokens[s]
        mean = (p * counts[s]).sum(1, keepdims=True)
        d, m = g * p * (counts[s] - mean), abs(g) * p * (counts[s] + mean)
        if score == "sigmoid":
            f = np.exp(-np.maximum(l[span], 0) - np.log1p(np.exp(-np.abs(l[span]))))   # 1 - sigma
            d, m = d * f, m * f
        grad[span], mag[span] = d, m
    return grad, mag
