"""Float64 CPU oracle of attention with modified scores: forward, backward and the
single-token step, written out from the definition in include/enc.h.

TEST INFRASTRUCTURE ONLY.  Shares no code with the CUDA library.  Dense: every
[batch, heads, queries, keys] array is formed, so it is meant for small sizes.

For query i and key j of a sequence with n valid positions, head h:
  u = scale q_i . k_j;  with a cap: u = cap tanh(u / cap)
  t = u - slopes[h] |j - i| + table[bucket(j - i)][h]
Key j is visible to query i where i, j < n, where causal asks for j <= i or
j < prefix, and where doc[i] == doc[j].  Rows that see nothing: ctx = 0,
lse = -inf.
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import Optional

import numpy as np


@dataclass
class ScoreSpec:
    scale: float
    cap: float = 0.0
    slopes: Optional[np.ndarray] = None        # [nh]
    table: Optional[np.ndarray] = None         # [num_buckets, nh]
    max_distance: int = 128
    bidirectional: bool = True
    causal: bool = False
    prefix_len: Optional[np.ndarray] = None    # [B]
    doc_ids: Optional[np.ndarray] = None       # [B, S]


def bucket(rel: int, num_buckets: int, max_distance: int, bidirectional: bool) -> int:
    """Bucket of the relative position rel = key - query."""
    m = num_buckets // 2 if bidirectional else num_buckets
    a = abs(rel) if bidirectional else max(-rel, 0)
    e = m // 2
    if a < e:
        c = a
    else:
        c = min(m - 1, e + math.floor(math.log(a / e) / math.log(max_distance / e) * (m - e) + 1e-9))
    return c + (m if bidirectional and rel > 0 else 0)


def bucket_matrix(spec: ScoreSpec, qpos, kpos) -> np.ndarray:
    nb = spec.table.shape[0]
    return np.array([[bucket(int(j) - int(i), nb, spec.max_distance, spec.bidirectional) for j in kpos] for i in qpos])


def bias(spec: ScoreSpec, nh: int, qpos, kpos) -> np.ndarray:
    """[nh, queries, keys]: the part of t that depends on the distance alone."""
    rel = np.asarray(kpos)[None, :] - np.asarray(qpos)[:, None]
    out = np.zeros((nh,) + rel.shape)
    if spec.slopes is not None:
        out -= spec.slopes.astype(np.float64)[:, None, None] * np.abs(rel)
    if spec.table is not None:
        out += np.moveaxis(spec.table.astype(np.float64)[bucket_matrix(spec, qpos, kpos)], -1, 0)
    return out


def visible(spec: ScoreSpec, valid_len, batch: int, seq: int) -> np.ndarray:
    """[B, S, S] truth values."""
    pos = np.arange(seq)
    n = np.clip(np.asarray(valid_len), 0, seq)
    ok = pos[None, :] < n[:, None]
    see = ok[:, :, None] & ok[:, None, :]
    if spec.causal:
        prefix = np.zeros(batch, int) if spec.prefix_len is None else np.asarray(spec.prefix_len)
        see &= (pos[None, None, :] <= pos[None, :, None]) | (pos[None, None, :] < prefix[:, None, None])
    if spec.doc_ids is not None:
        see &= spec.doc_ids[:, :, None] == spec.doc_ids[:, None, :]
    return see


def scores(spec: ScoreSpec, q, k, qpos, kpos):
    """(t, 1 - tanh^2) of q [B, nh, Sq, d] and k [B, nh, Sk, d]."""
    u = spec.scale * (q @ np.swapaxes(k, -1, -2))
    slope = np.ones_like(u)
    if spec.cap > 0:
        th = np.tanh(u / spec.cap)
        u, slope = spec.cap * th, 1 - th * th
    return u + bias(spec, q.shape[1], qpos, kpos)[None], slope


def _softmax(t, see):
    """P (zeros in rows that see nothing) and the log of the sum of exponentials."""
    t = np.where(see, t, -np.inf)
    top = t.max(-1, keepdims=True)
    e = np.exp(t - np.where(np.isfinite(top), top, 0.0))
    e = np.where(see, e, 0.0)
    total = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, np.where(np.isfinite(top), top, 0.0) + np.log(total), -np.inf)
    return e / np.where(total > 0, total, 1.0), lse[..., 0]


def _clean(x, valid_len, axis_seq):
    """x with the rows at or past the valid lengths (axis_seq; batch is axis 0) set to zero."""
    x = np.array(x, np.float64)
    moved = np.moveaxis(x, axis_seq, 1)
    for b, n in enumerate(np.clip(np.asarray(valid_len), 0, moved.shape[1])):
        moved[b, n:] = 0.0
    return x


def forward(spec: ScoreSpec, qkv, valid_len):
    """qkv [3, B, nh, S, d] -> ctx [B, S, nh, d], lse [B, nh, S], P [B, nh, S, S]."""
    _, B, nh, S, d = qkv.shape
    q, k, v = (_clean(qkv[i], valid_len, 2) for i in range(3))
    pos = np.arange(S)
    t, _ = scores(spec, q, k, pos, pos)
    p, lse = _softmax(t, visible(spec, valid_len, B, S)[:, None])
    return np.swapaxes(p @ v, 1, 2), lse, p


def backward(spec: ScoreSpec, qkv, valid_len, ctx, lse, dctx):
    """ctx and dctx [B, S, nh, d], lse [B, nh, S] -> dqkv [3, B, nh, S, d], dtable (None without a table),
    and (P, |P (dP - D)| bounds) for tolerances: P (|dctx| . |v| + |dctx| . |ctx|)."""
    _, B, nh, S, d = qkv.shape
    q, k, v = (_clean(qkv[i], valid_len, 2) for i in range(3))
    do = np.swapaxes(_clean(dctx, valid_len, 1), 1, 2)
    o = np.swapaxes(_clean(ctx, valid_len, 1), 1, 2)
    pos = np.arange(S)
    t, slope = scores(spec, q, k, pos, pos)
    see = visible(spec, valid_len, B, S)[:, None] & np.isfinite(lse)[..., None]
    p = np.where(see, np.exp(np.where(see, t, 0.0) - np.where(np.isfinite(lse), lse, 0.0)[..., None]), 0.0)
    dt = p * (do @ np.swapaxes(v, -1, -2) - (do * o).sum(-1, keepdims=True))
    size = p * (np.abs(do) @ np.swapaxes(np.abs(v), -1, -2) + (np.abs(do * o)).sum(-1, keepdims=True))
    du = dt * slope
    dq = spec.scale * (du @ k)
    dk = spec.scale * (np.swapaxes(du, -1, -2) @ q)
    dv = np.swapaxes(p, -1, -2) @ do
    dtable = None
    if spec.table is not None:
        dtable = np.zeros(spec.table.shape)
        np.add.at(dtable, bucket_matrix(spec, pos, pos), np.moveaxis(dt.sum(0), 0, -1))
    return np.stack((dq, dk, dv)), dtable, (p, size, du)


def step(spec: ScoreSpec, qkv, cache, length):
    """qkv [3, B, nh, 1, d], cache [2, B, nh, C, d], length [B] -> ctx [B, nh, d], cache after the step."""
    _, B, nh, C, d = cache.shape
    ctx, cache = np.zeros((B, nh, d)), np.array(cache)
    for b in range(B):
        p = int(length[b])
        if not 0 <= p < C:
            continue
        cache[0, b, :, p], cache[1, b, :, p] = qkv[1, b, :, 0], qkv[2, b, :, 0]
        t, _ = scores(spec, qkv[0, b:b + 1].astype(np.float64), cache[0, b:b + 1, :, :p + 1].astype(np.float64), [p],
                      np.arange(p + 1))
        see = np.ones(p + 1, bool) if spec.doc_ids is None else spec.doc_ids[b, :p + 1] == spec.doc_ids[b, p]
        pr, _ = _softmax(t, see[None, None, None, :])
        v = np.where(see[None, :, None], cache[1, b, :, :p + 1].astype(np.float64), 0.0)
        ctx[b] = (pr[0] @ v)[:, 0]
    return ctx, cache
