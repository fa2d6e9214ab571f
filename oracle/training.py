"""Oracle of the two ends of a tensor-parallel training step: dropout from a
counter-based generator on the way through a collective, and the softmax cross
entropy of a vocabulary cut over the ranks.

Dropout follows the library's stated arithmetic bit for bit (float32 fold,
scale, residual, one conversion).  The generator is Philox4x32-10 as its
authors publish it (Salmon, Moraes, Dror, Shaw: "Parallel random numbers: as
easy as 1, 2, 3", SC 2011).  The cross entropy is the definition in float64.
"""

import numpy as np

from .collectives import all_reduce_fold, chunk_bounds, from_acc, to_acc

_M = (np.uint64(0xD2511F53), np.uint64(0xCD9E8D57))
_W = (0x9E3779B9, 0xBB67AE85)
_LOW = np.uint64(0xFFFFFFFF)


def philox4x32(counter, key, rounds=10):
    """The four output words (uint32, last axis 4) for counters (..., 4) and a
    key of two words."""
    c = [np.asarray(counter, dtype=np.uint64)[..., i] for i in range(4)]
    k = [int(key[0]), int(key[1])]
    for _ in range(rounds):
        p0, p1 = _M[0] * c[0], _M[1] * c[2]
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), p1 & _LOW,
             (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), p0 & _LOW]
        k = [(k[0] + _W[0]) & 0xFFFFFFFF, (k[1] + _W[1]) & 0xFFFFFFFF]
    return np.stack(c, axis=-1).astype(np.uint32)


def dropout_keep(n, drop, seed, offset, start=0):
    """Which of the elements start .. start+n-1 stay."""
    i = np.arange(start, start + n, dtype=np.uint64)
    block = i // np.uint64(4)
    lo = block[0] if n else np.uint64(0)
    blocks = np.arange(int(lo), int(block[-1]) + 1 if n else 0, dtype=np.uint64)
    counter = np.zeros((blocks.size, 4), dtype=np.uint64)
    counter[:, 0] = blocks & _LOW
    counter[:, 1] = blocks >> np.uint64(32)
    counter[:, 2] = offset & 0xFFFFFFFF
    counter[:, 3] = (offset >> 32) & 0xFFFFFFFF
    words = philox4x32(counter, (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF)).reshape(-1)
    words = words[(i - lo * np.uint64(4)).astype(np.int64)] if n else words[:0]
    return words >= np.uint32(int(drop * 4294967296.0))


def _drop(values, keep, drop):
    scaled = values * np.float32(1.0 / (1.0 - drop))
    return np.where(keep, scaled, np.float32(0.0)).astype(np.float32)


def dropout(x, drop, seed, offset, dtype, residuals=None):
    """(p, n) inputs, rank by rank."""
    keep = dropout_keep(x.shape[1], drop, seed, offset)
    y = _drop(to_acc(x, dtype), keep[None, :], drop)
    if residuals is not None:
        y = y + to_acc(residuals, dtype)
    return from_acc(y, dtype)


def _fold32(x, dtype):
    """The ring-order fold before its conversion: float32."""
    return all_reduce_fold(to_acc(x, dtype), "sum", "float32")[0]


def all_reduce_dropout(x, drop, seed, offset, dtype, residuals=None):
    p, n = x.shape
    y = _drop(_fold32(x, dtype), dropout_keep(n, drop, seed, offset), drop)
    if residuals is None:
        return np.repeat(from_acc(y, dtype)[None, :], p, axis=0)
    return from_acc(y[None, :] + to_acc(residuals, dtype), dtype)


def reduce_scatter_dropout(x, drop, seed, offset, dtype, residuals=None):
    p, n = x.shape
    y = _drop(_fold32(x, dtype), dropout_keep(n, drop, seed, offset), drop).reshape(p, n // p)
    if residuals is not None:
        y = y + to_acc(residuals, dtype)
    return from_acc(y, dtype)


def all_gather_dropout(shards, drop, seed, offset, dtype):
    p = shards.shape[0]
    full = to_acc(shards, dtype).reshape(-1)
    y = from_acc(_drop(full, dropout_keep(full.size, drop, seed, offset), drop), dtype)
    return np.repeat(y[None, :], p, axis=0)


def vocab_shards(weight, p):
    b = chunk_bounds(weight.shape[0], p)
    return [weight[b[r]:b[r + 1]] for r in range(p)]


def cross_entropy(hidden, weight, targets, grad_loss=None):
    """Float64 (loss, lse) or (loss, lse, dhidden, dweight) of float64 hidden
    states [T, d] and the whole output weight [V, d]; a target outside [0, V)
    masks its token, whose hidden states then count for nothing."""
    vocab = weight.shape[0]
    live = (targets >= 0) & (targets < vocab)
    with np.errstate(invalid="ignore", over="ignore"):
        z = hidden @ weight.T
        top = z.max(axis=1, initial=-np.inf)
        lse = top + np.log(np.exp(z - top[:, None]).sum(axis=1))
    t = np.where(live, targets, 0)
    loss = np.where(live, lse - z[np.arange(z.shape[0]), t], 0.0)
    if grad_loss is None:
        return loss, lse
    rows = np.nonzero(live)[0]
    g = np.exp(z[rows] - lse[rows, None])
    g[np.arange(rows.size), targets[rows]] -= 1.0
    g *= np.asarray(grad_loss, dtype=np.float64)[rows, None]
    dhidden = np.zeros(hidden.shape)
    dhidden[rows] = g @ weight
    return loss, lse, dhidden, g.T @ hidden[rows]
