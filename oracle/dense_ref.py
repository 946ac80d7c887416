"""Plain float64 forms of the exact-attention operators (numpy, no code shared
with the GPU path), with the error that arithmetic of a given width may make.

Attention: S = scale q k^T; key j is visible to query i of batch b when
j < lens[b] and, if causal, j <= i + Nk - Nq; P = softmax over the visible
keys; O = P V; a row without a visible key has O = 0 and lse = -inf.  Query
head h reads key/value head h // (H // Hkv).
"""
from __future__ import annotations

import math

import numpy as np


def visible(B, Nq, Nk, causal=False, lens=None):
    """(B, 1, Nq, Nk) booleans."""
    j = np.arange(Nk)
    ok = np.ones((B, 1, Nq, Nk), bool)
    if lens is not None:
        ok &= (j < np.asarray(lens).reshape(B, 1, 1, 1))
    if causal:
        ok &= j <= np.arange(Nq)[:, None] + (Nk - Nq)
    return ok


def _shared(x, H):
    """Key/value heads repeated for the query heads that read them."""
    return np.repeat(x, H // x.shape[1], axis=1)


def _clean(x, lens):
    """x with zeros in the rows past each length (which may hold anything)."""
    if lens is None:
        return x
    x = x.copy()
    for b, n in enumerate(lens):
        x[b, :, max(0, min(int(n), x.shape[2])):] = 0
    return x


def _probabilities(q, k, scale, ok):
    S = np.where(ok, scale * q @ k.swapaxes(-1, -2), -np.inf)
    m = S.max(-1, keepdims=True, initial=-np.inf)
    m = np.where(np.isneginf(m), 0.0, m)
    E = np.exp(S - m)
    z = E.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (m + np.log(z))[..., 0]
    return E / np.where(z == 0, 1, z), lse


def dense_forward(q, k, v, causal=False, lens=None, scale=None):
    """(O, lse) of float64 (B, H, Nq, d) over (B, Hkv, Nk, d)."""
    B, H, Nq, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    k, v = (_shared(_clean(x, lens), H) for x in (k, v))
    P, lse = _probabilities(q, k, scale, visible(B, Nq, k.shape[2], causal, lens))
    return P @ v, lse


def dense_backward(q, k, v, dout, causal=False, lens=None, scale=None):
    """(dq, dk, dv) of sum(O dout)."""
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    kk, vv = (_shared(_clean(x, lens), H) for x in (k, v))
    P, _ = _probabilities(q, kk, scale, visible(B, Nq, Nk, causal, lens))
    dP = dout @ vv.swapaxes(-1, -2)
    dS = P * (dP - (P * dP).sum(-1, keepdims=True))

    def gather(x):  # sum over the query heads of a group
        return x.reshape(B, Hkv, H // Hkv, Nk, d).sum(2)

    return (scale * dS @ kk, gather(scale * dS.swapaxes(-1, -2) @ q),
            gather(P.swapaxes(-1, -2) @ dout))


def dense_errors(q, k, v, dout, half_step, causal=False, lens=None, scale=None,
                 rounded_weights=True, exact_delta=False):
    """Bounds on |error| of (O, lse, dq, dk, dv), element by element.

    half_step: finfo(dtype).eps / 2 of the tensors, by which every output is
    rounded once, and (rounded_weights) so are P before P V and P^T dO and dS
    before dS K and dS^T Q.  Everything else is fp32, where a sum of n terms
    is off by at most n eps32 times the sum of their magnitudes (eps32 = 2^-23
    covers truncating accumulators), and the exponential by 2^-21:
      p is off by e p,   e = 2 (d + 8) eps32 scale |q| |k|  + 2^-21 + Nk eps32
    (the score's error, twice for that of the row's log-sum-exp).  delta is
    taken from the rounded O, or, in the rows of exact_delta (one truth value, or
    (B, 1, Nq)), from the unrounded P and dP.
    """
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    eps = 2.0 ** -23
    scale = 1 / math.sqrt(d) if scale is None else scale
    kk, vv = (_shared(_clean(x, lens), H) for x in (k, v))
    ok = visible(B, Nq, Nk, causal, lens)
    P, lse = _probabilities(q, kk, scale, ok)
    a = np.where(ok, scale * np.abs(q) @ np.abs(kk).swapaxes(-1, -2), 0)
    worst = 2 * (d + 8) * eps * a.max(-1, keepdims=True, initial=0)
    e = worst + 2.0 ** -21 + Nk * eps
    w = half_step if rounded_weights else 0.0
    O = P @ vv
    eO = half_step * np.abs(O) + (w + e + Nk * eps) * (P @ np.abs(vv))
    eL = worst[..., 0] + 2.0 ** -21 + Nk * eps + eps * np.abs(np.where(np.isinf(lse), 0, lse))
    dP = dout @ vv.swapaxes(-1, -2)
    dS = P * (dP - (P * dP).sum(-1, keepdims=True))
    adP = np.abs(dout) @ np.abs(vv).swapaxes(-1, -2)
    eD = (np.abs(dout) * (eO + d * eps * np.abs(O))).sum(-1, keepdims=True)
    eP = ((e + Nk * eps) * P * np.abs(dP) + d * eps * P * adP).sum(-1, keepdims=True)
    eD = np.where(np.broadcast_to(exact_delta, (B, 1, Nq))[..., None], eP, eD)
    edS = (w + e) * np.abs(dS) + P * (d * eps * adP + eD)

    def gather(x):
        return x.reshape(B, Hkv, H // Hkv, Nk, d).sum(2)

    group = H // Hkv
    dq, dk, dv = dense_backward(q, k, v, dout, causal, lens, scale)
    n = (Nq * group + 4) * eps
    edq = half_step * np.abs(dq) + scale * (edS + (Nk + 4) * eps * np.abs(dS)) @ np.abs(kk)
    edk = half_step * np.abs(dk) + gather(
        scale * (edS + n * np.abs(dS)).swapaxes(-1, -2) @ np.abs(q))
    edv = half_step * np.abs(dv) + gather(((w + e + n) * P).swapaxes(-1, -2) @ np.abs(dout))
    return eO, eL, edq, edk, edv


def decode(q, k_cache, v_cache, table, lens, scale=None):
    """(O, lse, |P| |V|) of q (B, H, d) over paged caches (pages, Hkv, page_size, d)."""
    B, H, d = q.shape
    ps = k_cache.shape[2]
    scale = 1 / math.sqrt(d) if scale is None else scale
    O, A = np.zeros((B, H, d)), np.zeros((B, H, d))
    lse = np.full((B, H), -np.inf)
    rep = H // k_cache.shape[1]
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        rows = [(int(table[b, j // ps]), j % ps) for j in range(n)]
        K = np.stack([k_cache[p, :, r] for p, r in rows], 1)
        V = np.stack([v_cache[p, :, r] for p, r in rows], 1)
        for h in range(H):
            s = scale * K[h // rep] @ q[b, h]
            m = s.max()
            p = np.exp(s - m)
            lse[b, h] = m + math.log(p.sum())
            p /= p.sum()
            O[b, h], A[b, h] = p @ V[h // rep], p @ np.abs(V[h // rep])
    return O, lse, A


def rotary(x, positions, axis_dims, freqs, magnitude=1.0, interleaved=False, inverse=False):
    """Rotated (B, H, N, d); positions (B or 1, axes, N), freqs one per pair, axis after axis."""
    y = x.copy()
    at = r0 = 0
    for a, n in enumerate(axis_dims):
        for r in range(n // 2):
            i, j = (at + 2 * r, at + 2 * r + 1) if interleaved else (at + r, at + r + n // 2)
            t = np.asarray(positions, np.float64)[:, a][:, None] * freqs[r0 + r]
            t = -t if inverse else t
            y[..., i] = magnitude * (x[..., i] * np.cos(t) - x[..., j] * np.sin(t))
            y[..., j] = magnitude * (x[..., j] * np.cos(t) + x[..., i] * np.sin(t))
        at += n
        r0 += n // 2
    return y
