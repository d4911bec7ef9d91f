"""The operators whose rows have weights of their own (router, expert products, adapters) by their
definitions: what is defined step by step in binary32 is in binary32, the rest in 64 bits."""

import numpy as np
import torch

F32 = np.float32


def plan(owner, owners):
    """start, list of the items sorted by owner; a value outside [0, owners) means none."""
    owner = np.asarray(owner).reshape(-1)
    lists = [np.flatnonzero(owner == o) for o in range(owners)]
    start = np.concatenate([[0], np.cumsum([len(x) for x in lists])]).astype(np.int32)
    return start, np.concatenate(lists).astype(np.int32)


def topk(logits, k, bias=None, factor=1.0, sigmoid=False, norm=False):
    """logits: float64 array of what the row tensor holds. Returns expert, weight (64 bits)."""
    l32 = logits.astype(F32)
    score = l32 if bias is None else (l32 + bias.astype(F32)).astype(F32)
    live = score > -np.inf
    rows, experts = logits.shape
    expert = np.full((rows, k), -1, np.int32)
    weight = np.zeros((rows, k))
    for r in range(rows):
        order = sorted(np.flatnonzero(live[r]), key=lambda e: (-float(score[r, e]), e))[:k]
        if not order:
            continue
        expert[r, :len(order)] = order
        v = logits[r, order]
        with np.errstate(all="ignore"):
            if sigmoid:
                w = 1 / (1 + np.exp(-v))
                if norm:
                    w = w / w.sum() if w.astype(F32).sum() > 0 else 0 * w
            else:
                base = v if norm else logits[r, live[r]]
                w = np.exp(v - base.max()) / np.exp(base - base.max()).sum()
        weight[r, :len(order)] = w * factor
    return expert, weight


def codes(x):
    """int8 codes and scales of F32 rows, binary32 step by step; a row that is not finite: zeros and NaN."""
    x = x.astype(F32)
    fine = np.isfinite(x).all(1)
    amax = np.where(fine, np.abs(np.where(fine[:, None], x, 0)).max(1), 1).astype(F32)
    amax = np.maximum(amax, F32(1e-9))
    inv = (F32(127) / amax).astype(F32)
    v = np.clip((np.where(fine[:, None], x, F32(0)) * inv[:, None]).astype(F32).astype(np.float64), -127, 127)
    q = np.sign(v) * np.floor(np.abs(v) + 0.5)
    return q, np.where(fine, (amax / F32(127)).astype(F32), F32(np.nan)).astype(F32)


def dots(wq, bscale, owner, x, x_group):
    """d[item] in binary32 (zero for items without an expert); x: F32 rows."""
    q, scale = codes(x)
    d = np.zeros((owner.size, wq.shape[1]), F32)
    for e in range(wq.shape[0]):
        at = np.flatnonzero(owner == e)
        if at.size:
            row = at // x_group
            dot = (q[row] @ wq[e].astype(np.float64).T).astype(F32)   # exact below 2^53, rounded once
            d[at] = ((scale[row][:, None] * bscale[e][None]).astype(F32) * dot).astype(F32)
    return d


def swiglu(d):
    g, u = np.split(d.astype(np.float64), 2, 1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def swiglu_floor(d):
    """What binary32's range costs: exp(-g) is infinite from 88.7 on, where the result is then zero
    instead of |g u| 2^-128 at most, and results below the least normal number are off by half of 2^-149."""
    g, u = np.abs(np.split(d.astype(np.float64), 2, 1))
    return (g * 2.0 ** -127 + 2.0 ** -149) * u + 2.0 ** -149


def weighted(d, owner, experts, weight):
    rows, k = weight.shape
    d, here = d.reshape(rows, k, -1), ((owner >= 0) & (owner < experts)).reshape(rows, k)
    y = np.zeros((rows, d.shape[2]), F32)
    for j in range(k):
        with np.errstate(invalid="ignore"):
            y = np.where(here[:, j, None], (y + (weight[:, j, None] * d[:, j]).astype(F32)).astype(F32), y)
    return y


def lora(A, B, scale, owner, x, base):
    """out in 64 bits and the sums of the absolute values, t's and the outer product's (for the bounds)."""
    out, inner, outer = base.double().clone(), torch.zeros_like(base.double()), torch.zeros_like(base.double())
    for a in range(A.shape[0]):
        r = np.flatnonzero(owner == a)
        if r.size == 0:
            continue
        Ad, Bd, xd, s = A[a].double(), B[a].double(), x[r].double(), float(scale[a])
        t = xd @ Ad.T
        out[r] += s * (t @ Bd.T)
        inner[r] = abs(s) * ((xd.abs() @ Ad.abs().T) @ Bd.abs().T)
        outer[r] = abs(s) * (t.abs() @ Bd.abs().T)
    return out, inner, outer
