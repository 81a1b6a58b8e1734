"""Plain definitions of the serving operators around the cache: attention with a
sliding window and a few first tokens that stay visible, and the per-head norm with
the position rotation.

TEST INFRASTRUCTURE ONLY (see the package docstring): the CUDA library never imports
this module and this module never imports the library.

The pages stop at plain causal attention over a cache; these are the definitions
themselves, one loop per quantity, in float64:

* window: the query at position p sees key j when j <= p and (j > p - window or
  j < sinks).
* norm: y = x / sqrt(mean(x^2) + eps) * weight over one head's values.
* rotation: the pair (a, b) number i of the first ``rot`` values turns by the angle
  p * theta^(-2 i / rot); pairs are (i, i + rot / 2), or (2 i, 2 i + 1) interleaved.

Attention over a batch that shares a prefix needs no definition of its own: it is
``decode_paged`` over tables that name the shared blocks in every row.
"""

from __future__ import annotations

import numpy as np

from .attention import kv_head_for


def window_mask(Nq: int, Lk: int, window: int, sinks: int) -> np.ndarray:
    """Boolean ``[Nq, Lk]``: the ``Nq`` queries are the last positions of ``Lk`` tokens."""
    vis = np.zeros((Nq, Lk), dtype=bool)
    for t in range(Nq):
        p = Lk - Nq + t
        vis[t, max(0, p - window + 1):p + 1] = True
        vis[t, :min(sinks, p + 1)] = True
    return vis


def attention_window(q, k, v, scale, seqlens_k, window, sinks):
    """``q [B, Nq, Hq, d]``, ``k, v [B, Lcap, Hkv, d]`` -> ``o``, ``lse`` as ``attention``.

    Keys no query of the call sees are left out of the arithmetic (a cache may hold
    anything there)."""
    q = np.asarray(q, dtype=np.float64)
    B, Nq, Hq, d = q.shape
    Hkv = k.shape[2]
    o = np.zeros((B, Nq, Hq, d))
    lse = np.zeros((B, Hq, Nq))
    for b in range(B):
        L = int(seqlens_k[b])
        vis = window_mask(Nq, L, window, sinks)
        used = np.flatnonzero(vis.any(axis=0))
        vis = vis[:, used]
        for h in range(Hq):
            g = kv_head_for(h, Hq, Hkv)
            kk = np.asarray(k[b, used, g], dtype=np.float64)
            vv = np.asarray(v[b, used, g], dtype=np.float64)
            s = np.where(vis, scale * (q[b, :, h] @ kk.T), -np.inf)
            m = s.max(axis=1, keepdims=True)
            w = np.exp(s - m)
            z = w.sum(axis=1, keepdims=True)
            o[b, :, h] = (w @ vv) / z
            lse[b, h] = (m + np.log(z))[:, 0]
    return o, lse


def head_norm(x, weight, eps):
    """``x [..., d]`` normalised over its last axis; no weight, no norm."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x.copy()
    return x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)


def rotate(y, positions, rot, theta=10000.0, interleaved=False):
    """``y [B, T, H, d]`` turned at ``positions [B, T]``, first ``rot`` values of each head."""
    y = np.array(y, dtype=np.float64, copy=True)
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        angle = np.asarray(positions, dtype=np.float64)[:, :, None] * theta ** (-2.0 * i / rot)
        c, s = np.cos(angle), np.sin(angle)
        ya, yb = y[..., a].copy(), y[..., b].copy()
        y[..., a] = ya * c - yb * s
        y[..., b] = yb * c + ya * s
    return y


def norm_rotate(x, weight, eps, positions, rot, theta=10000.0, interleaved=False):
    return rotate(head_norm(x, weight, eps), positions, rot, theta, interleaved)
