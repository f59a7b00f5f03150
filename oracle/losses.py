"""Plain fp64 losses of a linear head on the CPU (numpy), with their gradients.

Everything is computed from the definitions over the whole logit matrix; the
split of the vocabulary over ranks only decides which rows of W (and of dW)
belong to whom, so W here is the whole head [V, D].
"""
from __future__ import annotations

import numpy as np


def logits(X, W, softcap=0.0):
    """l = X W^T, capped by softcap * tanh(x / softcap) when softcap > 0."""
    x = np.asarray(X, np.float64) @ np.asarray(W, np.float64).T
    return softcap * np.tanh(x / softcap) if softcap else x


def logsumexp(l):
    m = l.max(axis=1, keepdims=True)
    return (m + np.log(np.exp(l - m).sum(axis=1, keepdims=True)))[:, 0]


def xent(X, W, labels, ignore_index=-100, smoothing=0.0, z_weight=0.0, softcap=0.0):
    """(loss, lse), one of each per token; ignored and impossible labels give loss 0."""
    l = logits(X, W, softcap)
    lse = logsumexp(l)
    loss = np.zeros(len(l))
    for t, y in enumerate(labels):
        if y != ignore_index and 0 <= y < l.shape[1]:
            loss[t] = (lse[t] - (1 - smoothing) * l[t, y] - smoothing * l[t].mean()
                       + z_weight * lse[t] ** 2)
    return loss, lse


def xent_dlogits(X, W, labels, dloss, ignore_index=-100, smoothing=0.0, z_weight=0.0,
                 softcap=0.0):
    """Gradient of sum_t dloss_t loss_t with respect to the uncapped logits X W^T."""
    l = logits(X, W, softcap)
    lse = logsumexp(l)
    d = np.zeros_like(l)
    for t, y in enumerate(labels):
        if y == ignore_index or not 0 <= y < l.shape[1]:
            continue
        d[t] = (1 + 2 * z_weight * lse[t]) * np.exp(l[t] - lse[t]) - smoothing / l.shape[1]
        d[t, y] -= 1 - smoothing
        d[t] *= dloss[t]
        if softcap:
            d[t] *= 1 - (l[t] / softcap) ** 2
    return d


def teacher_probs(idx, teacher, V, temperature):
    """Per token: the list of (vocabulary index, probability) of its valid entries."""
    rows = []
    for t in range(len(idx)):
        at = [k for k in range(idx.shape[1])
              if 0 <= idx[t, k] < V and teacher[t, k] != -np.inf]
        if not at:
            rows.append([])
            continue
        x = np.asarray([float(teacher[t, k]) for k in at])
        e = np.exp((x - x.max()) / temperature)
        rows.append([(int(idx[t, k]), q) for k, q in zip(at, e / e.sum())])
    return rows


def distill(X, W, idx, teacher, temperature=1.0, softcap=0.0):
    """(loss, lse) of the distillation from the teacher's top logits."""
    l = logits(X, W, softcap) / temperature
    lse = logsumexp(l)
    loss = np.zeros(len(l))
    for t, row in enumerate(teacher_probs(idx, teacher, l.shape[1], temperature)):
        if row:
            loss[t] = temperature ** 2 * (
                sum(q * (np.log(q) - l[t, i]) for i, q in row if q > 0) + lse[t])
    return loss, lse


def distill_dlogits(X, W, idx, teacher, dloss, temperature=1.0, softcap=0.0):
    l = logits(X, W, softcap)
    lse = logsumexp(l / temperature)
    d = np.zeros_like(l)
    for t, row in enumerate(teacher_probs(idx, teacher, l.shape[1], temperature)):
        if not row:
            continue
        d[t] = np.exp(l[t] / temperature - lse[t])
        for i, q in row:
            d[t, i] -= q
        d[t] *= dloss[t] * temperature
        if softcap:
            d[t] *= 1 - (l[t] / softcap) ** 2
    return d


def gradients(dlogits, X, W):
    """(dX, dW) of the uncapped logits' gradient."""
    return dlogits @ np.asarray(W, np.float64), dlogits.T @ np.asarray(X, np.float64)
