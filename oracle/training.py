"""Oracle of the training operators — TEST INFRASTRUCTURE ONLY (numpy, float64).

Dropout from a counter-based generator, dropout + residual + LayerNorm and its
backward, the gated linear unit and its backward, the weight gradient.  Plain
definitions in 64 bits, pinned by ``tests/test_training_oracle.py`` (published
vectors of the generator, finite differences, torch in float64).
"""
from __future__ import annotations

import math

import numpy as np

# Philox4x32-10: Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as 1, 2, 3" (SC 2011)
PHILOX_M = (0xD2511F53, 0xCD9E8D57)
PHILOX_W = (0x9E3779B9, 0xBB67AE85)
_LOW = np.uint64(0xFFFFFFFF)
_SH = np.uint64(32)


def philox4x32(ctr, key, rounds: int = 10) -> np.ndarray:
    """ctr: four uint32 arrays (or numbers) of one shape, key: two numbers -> [..., 4] uint32."""
    c = [np.asarray(x, dtype=np.uint64) for x in np.broadcast_arrays(*ctr)]
    k = [int(x) for x in key]
    for _ in range(rounds):
        p0, p1 = c[0] * np.uint64(PHILOX_M[0]), c[2] * np.uint64(PHILOX_M[1])
        c = [(p1 >> _SH) ^ c[1] ^ np.uint64(k[0]), p1 & _LOW, (p0 >> _SH) ^ c[3] ^ np.uint64(k[1]), p0 & _LOW]
        k = [(k[0] + PHILOX_W[0]) & 0xFFFFFFFF, (k[1] + PHILOX_W[1]) & 0xFFFFFFFF]
    return np.stack(c, axis=-1).astype(np.uint32)


def keep_mask(M: int, N: int, p: float, seed: int, offset: int) -> np.ndarray:
    """True where element (m, n) is kept: word n mod 4 of the block m·⌈N/4⌉ + n/4 is at least ⌊p·2^32⌋
    (p as a 32-bit float; seed and offset modulo 2^64)."""
    p = float(np.float32(p))
    seed, offset = seed % 2**64, offset % 2**64
    g = -(-N // 4)
    block = np.arange(M * g, dtype=np.uint64)
    r = philox4x32((block & _LOW, block >> _SH, np.uint64(offset & 0xFFFFFFFF), np.uint64(offset >> 32)),
                   (seed & 0xFFFFFFFF, seed >> 32))
    return (r >= np.uint32(math.floor(p * 2.0**32))).reshape(M, 4 * g)[:, :N]


def dropout(x, p: float, seed: int, offset: int) -> np.ndarray:
    x = np.asarray(x, np.float64)
    if p == 0.0:
        return x
    return np.where(keep_mask(*x.shape, p, seed, offset), x / (1.0 - float(np.float32(p))), 0.0)


def dropout_layernorm(x, residual, gamma, beta, eps, p=0.0, seed=0, offset=0):
    """(s, z, mean, rstd), nothing rounded."""
    s = dropout(x, p, seed, offset)
    if residual is not None:
        s = s + residual
    mean = s.mean(axis=1)
    d = s - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + eps)
    z = d * rstd[:, None]
    if gamma is not None:
        z = z * gamma
    if beta is not None:
        z = z + beta
    return s, z, mean, rstd


def dropout_layernorm_backward(dz, dsum, s, mean, rstd, gamma, p=0.0, seed=0, offset=0):
    """(dres, dx, dgamma, dbeta), nothing rounded."""
    u = (s - mean[:, None]) * rstd[:, None]
    g = dz if gamma is None else dz * gamma
    ds = rstd[:, None] * (g - g.mean(axis=1, keepdims=True) - u * (g * u).mean(axis=1, keepdims=True))
    if dsum is not None:
        ds = ds + dsum
    return ds, dropout(ds, p, seed, offset), (dz * u).sum(axis=0), dz.sum(axis=0)


def _logistic(kind: str, v: np.ndarray):
    """(σ(y), σ(-y), y') of the gate v·σ(y).  SWIGLU: y = v.  GEGLU_TANH: (1 + tanh w)/2 = σ(2w), so y = 2w with
    w = √(2/π)·(v + 0.044715·v³); in this form nothing cancels where tanh w is near -1."""
    if kind == "SWIGLU":
        y, dy = v, np.ones_like(v)
    else:
        c = 2.0 * math.sqrt(2.0 / math.pi)
        y, dy = c * (v + 0.044715 * v**3), c * (1.0 + 3.0 * 0.044715 * v * v)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-y)), 1.0 / (1.0 + np.exp(y)), dy


def gate(v, kind: str) -> np.ndarray:
    """The gate's activation: v·σ(v) (SWIGLU) or the tanh GELU (GEGLU_TANH)."""
    v = np.asarray(v, np.float64)
    return v * _logistic(kind, v)[0]


def gate_grad(v, kind: str) -> np.ndarray:
    v = np.asarray(v, np.float64)
    s, t, dy = _logistic(kind, v)
    return s + v * s * t * dy


def glu(x, W, kind: str):
    """(h, gu): gu = x·Wᵀ for the stacked W = [Wg; Wu], h = gate(g)·u."""
    gu = np.asarray(x, np.float64) @ np.asarray(W, np.float64).T
    N = gu.shape[1] // 2
    return gate(gu[:, :N], kind) * gu[:, N:], gu


def glu_backward(dy, Wd, gu, kind: str):
    """(dgu, dh): dh = dy·Wd for the down weight Wd [K, N]; dgu = [dh·u·gate'(g), dh·gate(g)]."""
    dh = np.asarray(dy, np.float64) @ np.asarray(Wd, np.float64)
    N = dh.shape[1]
    g, u = gu[:, :N], gu[:, N:]
    return np.concatenate([dh * u * gate_grad(g, kind), dh * gate(g, kind)], axis=1), dh


def weight_grad(dy, x, before=None, scale: float = 1.0) -> np.ndarray:
    """(dyᵀ·x + before)·scale for dy [tokens, out] and x [tokens, in]."""
    dw = np.asarray(dy, np.float64).T @ np.asarray(x, np.float64)
    return (dw if before is None else dw + before) * scale
