"""fp64 oracle of attention on packed plain rows with a learned relative position bias, and of its gradient.

Plain numpy on the definition; shares no code with the kernels.
"""
from __future__ import annotations

import numpy as np


def first_distances(num_buckets: int, max_distance: int) -> list[int]:
    """Smallest distance of each bucket.  With m = num_buckets // 2 and r = num_buckets - m, distance n >= m
    lies in bucket m + floor(r ln(n / m) / ln(max_distance / m)) or beyond it exactly when
    n^r >= m^(r - j) max_distance^j, which whole numbers decide."""
    m = num_buckets // 2
    r = num_buckets - m
    first = list(range(m))
    n = m
    for j in range(r):
        while n ** r < m ** (r - j) * max_distance ** j:
            n += 1
        first.append(n)
    return first


def buckets(distances, num_buckets: int, max_distance: int) -> np.ndarray:
    return np.searchsorted(first_distances(num_buckets, max_distance), np.maximum(distances, 0), side="right") - 1


def _ij(x, y):
    """[h, i, j] = sum over d of x[i, h, d] y[j, h, d]."""
    return x.transpose(1, 0, 2) @ y.transpose(1, 2, 0)


def _rows(w, x):
    """[i, h, d] = sum over j of w[h, i, j] x[j, h, d]."""
    return (w @ x.transpose(1, 0, 2)).transpose(1, 0, 2)


def _sequence(q, k, window, scale, bias, max_distance):
    """Weights [H, sq, sk], lse [H, sq], the mask and the distances of one sequence (q [sq, H, D], k [sk, Hkv, D])."""
    sq, heads, _ = q.shape
    sk, hkv, _ = k.shape
    kk = np.repeat(k, heads // hkv, axis=1)
    s = _ij(q, kk) * scale
    far = (sk - sq + np.arange(sq))[:, None] - np.arange(sk)[None]
    see = (far >= 0) & ((far < window) if window > 0 else True)
    if bias is not None and sk > 0:
        s = s + bias[buckets(far, bias.shape[0], max_distance)].transpose(2, 0, 1)
    s = np.where(see, s, -np.inf)
    top = s.max(axis=-1, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0)[..., None])
    total = e.sum(-1)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, np.where(np.isfinite(top), top, 0.0) + np.log(total), -np.inf)
    return e / np.where(total > 0, total, 1.0)[..., None], lse, see, far, np.where(np.isfinite(s), np.abs(s), 0.0)


def attention(q, k, v, cu_q, cu_k, window=0, scale=1.0, bias=None, max_distance=0, dout=None):
    """Packed attention in fp64; with dout its gradient too.  Returns a dict of arrays; rows outside every sequence are
    NaN.  `out_abs`, and for the gradients `*_abs` and `*_terms`, are the sums of the absolute terms that error
    bounds need: out_abs = sum P |v|, and with N = |dout| |v|^T, M = sum_j P N:
    dq_abs = scale sum |dS| |k|, dq_terms = scale sum P (N + M) |k|, dq_rows = scale sum P |k|; likewise for dk (and
    dv_abs = sum P |dout|, dbias_terms = sum P (N + M) + |dS| by bucket)."""
    heads, hkv = q.shape[1], k.shape[1]
    g = heads // hkv
    nan = lambda shape: np.full(shape, np.nan)  # noqa: E731
    r = {"out": nan(q.shape), "lse": nan(q.shape[:2]), "out_abs": nan(q.shape), "logit": np.zeros(q.shape[:2])}
    if dout is not None:
        for n, like in (("dq", q), ("dk", k), ("dv", k)):
            for e in ("", "_abs", "_terms", "_rows"):
                r[n + e] = nan(like.shape)
        if bias is not None:
            r["dbias"], r["dbias_terms"] = np.zeros(bias.shape), np.zeros(bias.shape)
    for a, b, c, d in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        qi, ki, vi = q[a:b], k[c:d], v[c:d]
        p, lse, see, far, size = _sequence(qi, ki, window, scale, bias, max_distance)
        vv, kk = np.repeat(vi, g, axis=1), np.repeat(ki, g, axis=1)
        r["out"][a:b] = _rows(p, vv)
        r["out_abs"][a:b] = _rows(p, np.abs(vv))
        r["lse"][a:b] = lse.T
        r["logit"][a:b] = (_ij(np.abs(qi), np.abs(kk)) * scale * see + size).max(-1, initial=0.0).T
        if dout is None:
            continue
        do = dout[a:b]
        dp = _ij(do, vv)
        n = _ij(np.abs(do), np.abs(vv))
        ds = p * (dp - (p * dp).sum(-1, keepdims=True))
        terms = p * (n + (p * n).sum(-1, keepdims=True))
        share = lambda x: x.reshape(x.shape[0], hkv, g, x.shape[2]).sum(2)  # noqa: E731
        r["dq"][a:b] = scale * _rows(ds, kk)
        r["dk"][c:d] = scale * share(_rows(ds.transpose(0, 2, 1), qi))
        r["dv"][c:d] = share(_rows(p.transpose(0, 2, 1), do))
        r["dv_abs"][c:d] = share(_rows(p.transpose(0, 2, 1), np.abs(do)))
        for e, w in (("_abs", np.abs(ds)), ("_terms", terms), ("_rows", p)):
            r["dq" + e][a:b] = scale * _rows(w, np.abs(kk))
            r["dk" + e][c:d] = scale * share(_rows(w.transpose(0, 2, 1), np.abs(qi)))
        if bias is not None and d > c:
            by = buckets(far, bias.shape[0], max_distance)
            for i in range(bias.shape[0]):
                hit = see & (by == i)
                r["dbias"][i] += (ds * hit).sum((1, 2))
                r["dbias_terms"][i] += ((terms + np.abs(ds)) * hit).sum((1, 2))
    return r
