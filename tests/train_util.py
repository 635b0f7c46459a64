"""Helpers for the training-step operator tests: seeded tensors, their exact
values, and error bounds.

Unit roundoffs (half a step, relative): f32 2^-24, f16 2^-11 and bf16 2^-8 as
bounds on one rounding; a sum of n f32 terms in any order is off by at most
(n - 1) 2^-24 / (1 - n 2^-24) times the sum of the magnitudes.  The matrix
instructions are not promised to round each addition to nearest, so their sums
count twice that (one unit instead of half a unit per addition)."""

import numpy as np
import torch

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
U32 = 2.0 ** -24
ROUND = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}   # smallest step


def rng(*key):
    return np.random.default_rng([20261206, *key])


def tensor(a, dtype, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(DTYPES[dtype]).to(device)


def exact(t):
    """A tensor's values in float64."""
    return t.detach().to("cpu").double().numpy()


def shards(vocab, ranks):
    block = -(-vocab // ranks)
    return [max(0, min(block, vocab - r * block)) for r in range(ranks)]


def sum_bound(n):
    """Relative to the sum of magnitudes: n terms added on the matrix cores."""
    return 2.0 * (n + 2) * U32


def worst(got, want, tol):
    """The largest |got - want| / tol, infinite for a misplaced NaN."""
    got, want, tol = np.broadcast_arrays(got, want, tol)
    if got.size == 0:
        return 0.0
    if not np.array_equal(np.isfinite(got), np.isfinite(want)):
        return np.inf
    ok = np.isfinite(want)
    return float((np.abs(got[ok] - want[ok]) / tol[ok]).max()) if ok.any() else 0.0


def xent_bounds(x, ws, targets, lse, dloss, dtype):
    """Bounds on the errors of (loss, lse, dx, dw), from the definition:

    a logit is off by dz = sum_bound(dim) * |x| . |w|; exp2(y log2 e) of y = z -
    m takes two roundings of y (|y| 2^-23 absolute in the exponent) and the
    instruction's own 2^-22; a sum over the vocabulary adds V terms; log and
    the last addition round once each."""
    from oracle import train as O
    w = np.concatenate(ws)
    z, size = x @ w.T, np.abs(x) @ np.abs(w).T
    dz = sum_bound(x.shape[1]) * size + 2.0 ** -149
    spread = np.abs(z - z.max(1, keepdims=True))
    p = O.softmax_rows(z)
    rel = (p * (dz + dz.max(1, keepdims=True) + spread * 4 * U32)).sum(1) + (z.shape[1] + 16) * U32
    lse_tol = rel + 4 * U32 * (1 + np.abs(z).max(1) + np.abs(lse))
    ok = O.counted(targets, len(w))
    at = dz[np.arange(len(targets)), np.where(ok, targets, 0)]
    loss_tol = lse_tol + at + 4 * U32 * np.abs(z).max(1)
    g = O.logit_gradient(x, ws, targets, lse, dloss)
    q = np.exp(np.minimum(z - lse[:, None], 80.0))
    dg = np.abs(dloss)[:, None] * q * (dz + (np.abs(z - lse[:, None]) + 4) * 4 * U32) + np.abs(g) * 4 * U32
    dg[~ok] = 0.0
    # stored in the buffer type: f32 as it is, 16-bit types as q = g / dloss
    # (f16: times 2^14, so that its smallest step is 2^-24 / 2^14 of |dloss|); up
    # to 64 tokens g / top as hi + lo: half a step of lo, which is half a step of
    # hi or less
    top = np.abs(dloss[ok]).max() if ok.any() else 0.0
    two = dtype != "f32" and len(x) <= 64
    stored = ROUND[dtype] ** 2 + 4 * U32 if two else ROUND[dtype]
    dg += np.abs(g) * stored + (top * 2.0 ** -38 if dtype == "f16" else TINY[dtype] * max(1.0, top))
    dg[~ok] = 0.0
    xs = np.where(ok[:, None], np.abs(x), 0.0)
    size_dx, size_dw = np.abs(g) @ np.abs(w), np.abs(g).T @ xs
    # a 16-bit dx is multiplied by dloss (one rounding in f32); hi and lo are
    # summed apart, their magnitudes at most 1 + ROUND of the whole
    twice = 1 + 2 * ROUND[dtype] if two else 1.0
    dx_tol = dg @ np.abs(w) + (twice * sum_bound(len(w)) + 3 * U32) * size_dx
    dw_tol = dg.T @ xs + twice * sum_bound(2 * len(x)) * size_dw
    if dtype != "f32" and not two:
        # x' = x dloss / top: two roundings in f32, one to the type (half of its
        # smallest step where that is more); dw is multiplied by top (over 2^14)
        dw_tol += (ROUND[dtype] + 4 * U32) * size_dw + TINY[dtype] / 2 * top * q[ok].sum(0)[:, None] + TINY[dtype] * top * len(x)
    return loss_tol, lse_tol, dx_tol, dw_tol


def rounded(want, tol, dtype):
    """`tol` before the last rounding to dtype, with that rounding."""
    return tol * (1 + ROUND[dtype]) + np.abs(want) * ROUND[dtype] + TINY[dtype]


def emulated_ortho(g, steps, coeffs, dtype):
    """The library's number formats on the host: X as hi + lo f16 pairs times
    1024, factors as pairs (bf16: hi alone), products in f32."""
    pair = dtype != "bf16"

    def split(v):
        v = (v * np.float32(1024)).astype(np.float32)
        hi = v.astype(np.float16).astype(np.float32)
        return hi, (v - hi).astype(np.float16).astype(np.float32)

    def mul(p, q):
        s = p[0] @ q[0]
        if pair:
            s = s + (p[1] @ q[0] + p[0] @ q[1])
        return s * np.float32(2.0 ** -20)

    def value(p, whole=True):
        return (p[0] + p[1] if whole else p[0]) / np.float32(1024)

    tall = g.shape[0] > g.shape[1]
    x = g.T if tall else g
    x = split((x / (np.sqrt((x * x).sum()) + 1e-7)).astype(np.float32))
    for a, b, c in coeffs:
        a, b, c = np.float32(a), np.float32(b), np.float32(c)
        gram = split(mul(x, (x[0].T, x[1].T)))
        poly = split(b * value(gram, pair) + c * mul(gram, gram))
        x = split(a * value(x) + mul(poly, x))
    x = value(x).astype(np.float64)
    return x.T if tall else x
