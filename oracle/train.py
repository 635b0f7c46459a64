"""Plain 64-bit implementations of the training-step operators: softmax cross
entropy with the vocabulary split over ranks, the balance loss of a
mixture-of-experts router, and Newton-Schulz orthogonalisation.  Inputs are
float64 arrays that hold the buffers' values exactly; nothing is rounded.
"""

from __future__ import annotations

import numpy as np

DEFAULT_COEFFS = (3.4445, -4.7750, 2.0315)


def counted(targets, vocab):
    """Which tokens have a loss: those whose target is a row of the vocabulary."""
    return (targets >= 0) & (targets < vocab)


def cross_entropy(x, ws, targets):
    """(loss, lse) of hidden states against the ranks' rows laid end to end."""
    z = x @ np.concatenate(ws).T
    top = z.max(1)
    ref = np.where(np.isfinite(top), top, 0.0)
    with np.errstate(divide="ignore"):
        lse = ref + np.log(np.exp(z - ref[:, None]).sum(1))
    ok = counted(targets, z.shape[1])
    at = z[np.arange(len(targets)), np.where(ok, targets, 0)]
    return np.where(ok, lse - at, 0.0), lse


def logit_gradient(x, ws, targets, lse, dloss):
    """d L / d logits, zeros in the rows of tokens without a loss."""
    z = x @ np.concatenate(ws).T
    ok = counted(targets, z.shape[1])
    g = np.zeros_like(z)
    g[ok] = np.exp(z[ok] - lse[ok, None])
    rows = np.flatnonzero(ok)
    g[rows, targets[rows]] -= 1.0
    return g * np.where(ok, dloss, 0.0)[:, None]


def cross_entropy_grad(x, ws, targets, lse, dloss):
    """(dx, [dw of every rank]); a token without a loss takes no part."""
    g = logit_gradient(x, ws, targets, lse, dloss)
    ok = counted(targets, g.shape[1])
    dw = g[ok].T @ x[ok]
    dx = np.zeros_like(x)
    dx[ok] = g[ok] @ np.concatenate(ws)
    return dx, np.split(dw, np.cumsum([len(w) for w in ws])[:-1])


def softmax_rows(z):
    """Row softmax; a row of -infinities has no probabilities (zeros)."""
    top = z.max(1, keepdims=True)
    p = np.exp(z - np.where(np.isneginf(top), 0.0, top))
    s = p.sum(1, keepdims=True)
    return np.divide(p, s, out=np.zeros_like(p), where=s != 0)


def balance_loss(logits, experts, coef):
    """(counts [ranks + 1, E], loss, [gradient of every rank's logits])."""
    nexp, topk = logits[0].shape[1], experts[0].shape[1]
    counts = np.zeros((len(logits) + 1, nexp), np.int64)
    live, probs = [], []
    for r, (z, idx) in enumerate(zip(logits, experts)):
        ok = (idx >= 0) & (idx < nexp)
        np.add.at(counts[r], idx[ok], 1)
        live.append(ok.any(1))
        p = np.zeros_like(z)
        p[live[-1]] = softmax_rows(z[live[-1]]) if live[-1].any() else 0.0
        probs.append(p)
    counts[-1] = counts[:-1].sum(0)
    n = int(sum(v.sum() for v in live))
    if n == 0:
        return counts, 0.0, [np.zeros_like(z) for z in logits]
    f = counts[-1] / (n * topk)
    mean = sum(p.sum(0) for p in probs) / n
    grads = [coef * nexp / n * p * (f - (p @ f)[:, None]) for p in probs]
    return counts, coef * nexp * float(f @ mean), grads


def orthogonalize(g, steps, coeffs=None):
    """Newton-Schulz steps on g / (|g| + 1e-7); ``coeffs``: a triple per step."""
    coeffs = [DEFAULT_COEFFS] * steps if coeffs is None else coeffs
    tall = g.shape[0] > g.shape[1]
    x = g.T if tall else g
    x = x / (np.sqrt((x * x).sum()) + 1e-7)
    for a, b, c in coeffs:
        gram = x @ x.T
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.T if tall else x
