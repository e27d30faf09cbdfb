"""Packed attention for tests: 64-bit values and error terms in torch (on the GPU, for sequences too long for numpy), and which
blocks of the gradient's dK/dV kernel take which parts of which key tiles.  Shares no code with the kernels.

Error terms as in oracle/relative.py: N = |dout| |v|^T; `out_abs` = sum P |v|, `*_abs` the sums of |dS| (dv: of P) times the
absolute operand, `*_terms` those of P (N + sum P N), `*_rows` those of P.
"""
import os
import re

import numpy as np
import torch

from oracle import relative

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_attention_03_gb300", "csrc")


def values(q, k, v, cu_q, cu_k, window, scale, bias=None, max_distance=0, dout=None):
    """A dict as oracle.relative.attention's, of float64 tensors on q's device; and `ds_abs` [Tq, H] = sum_j |dS_ij|,
    `mean` [Tq, H] = sum_j P_ij N_ij."""
    d = q.device
    wide = lambda t: torch.zeros(t.shape, dtype=torch.float64, device=d)  # noqa: E731
    heads, hkv = q.shape[1], k.shape[1]
    group = heads // hkv
    r = {"out": wide(q), "out_abs": wide(q), "lse": wide(q[..., 0]), "logit": wide(q[..., 0])}
    if dout is not None:
        r |= {"ds_abs": wide(q[..., 0]), "mean": wide(q[..., 0])}
        r |= {n + e: wide(like) for n, like in (("dq", q), ("dk", k), ("dv", v)) for e in ("", "_abs", "_terms", "_rows")}
        if bias is not None:
            r |= {"dbias": wide(bias), "dbias_terms": wide(bias)}
    for a, b, c, e in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        a, b, c, e = int(a), int(b), int(c), int(e)
        if a == b:
            continue
        far = (e - c) - (b - a) + torch.arange(b - a, device=d)[:, None] - torch.arange(e - c, device=d)
        hide = far < 0
        if window > 0:
            hide = hide | (far >= window)
        if bias is not None:
            by = torch.as_tensor(relative.buckets(np.arange(max(e - c, 1)), bias.shape[0], max_distance), device=d)
        for h in range(heads):
            g = h // group
            x, y, z = q[a:b, h].double(), k[c:e, g].double(), v[c:e, g].double()
            s = scale * (x @ y.T)
            size = scale * (x.abs() @ y.abs().T)
            if bias is not None and e > c:
                add = bias[:, h].double()[by[far.clamp(min=0)]]
                s, size = s + add, size + add.abs().nan_to_num(posinf=0.0)
            s = s.masked_fill(hide, float("-inf"))
            r["logit"][a:b, h] = size.masked_fill(torch.isinf(s), 0.0).amax(1) if e > c else 0.0
            r["lse"][a:b, h] = torch.logsumexp(s, 1)
            p = torch.exp(s - r["lse"][a:b, h, None]).nan_to_num(nan=0.0)  # (a row without keys has none)
            r["out"][a:b, h], r["out_abs"][a:b, h] = p @ z, p @ z.abs()
            if dout is None:
                continue
            o = dout[a:b, h].double()
            dp, n = o @ z.T, o.abs() @ z.abs().T
            ds = p * (dp - (p * dp).sum(1, keepdim=True))
            terms = p * (n + (p * n).sum(1, keepdim=True))
            r["ds_abs"][a:b, h], r["mean"][a:b, h] = ds.abs().sum(1), (p * n).sum(1)
            r["dq"][a:b, h] = scale * (ds @ y)
            r["dk"][c:e, g] += scale * (ds.T @ x)
            r["dv"][c:e, g] += p.T @ o
            r["dv_abs"][c:e, g] += p.T @ o.abs()
            for kind, w in (("_abs", ds.abs()), ("_terms", terms), ("_rows", p)):
                r["dq" + kind][a:b, h] = scale * (w @ y.abs())
                r["dk" + kind][c:e, g] += scale * (w.T @ x.abs())
            if bias is not None and e > c:
                index = by[far.clamp(min=0)].flatten()
                for name, w in (("dbias", ds), ("dbias_terms", terms + ds.abs())):
                    r[name][:, h].index_add_(0, index, w.masked_fill(hide, 0.0).flatten())
    return r


def constant(name, file):
    with open(os.path.join(CSRC, file)) as f:
        return int(re.search(r"\b%s = (\d+)" % name, f.read()).group(1))


def key_items(sq, sk, heads, hkv, window=0, sms=152):
    """The dK/dV kernel's work by block: for each, the list of (key tile, part, parts, kv head) that it takes in turn.  Tiles of 128 keys
    have a step for each head of the kv head and each 128 queries that see some of them, tiles of more steps than an SM's share
    and a few are split, and the parts, longest first, are dealt with their kv heads in snake order."""
    group, tiles = heads // hkv, []
    for q, k in zip(sq, sk):
        for t in range(-(-k // 128)):
            first = max(0, 128 * t - (k - q))
            end = q if window <= 0 else min(q, 128 * t + min(k - 128 * t, 128) - 1 + window - (k - q))
            tiles.append(max(0, -(-(end - first) // 128)) * group)
    limit = sum(tiles) * hkv // sms + constant("kMinSteps", "attn_backward.cu")
    entries = []
    for i, steps in enumerate(tiles):
        parts = max(-(-steps // limit), 1)
        per = -(-steps // parts)
        entries += [(min(per * (p + 1), steps) - per * p, i, p, parts) for p in range(parts)]
    entries.sort(key=lambda x: -x[0])
    items = [(i, p, parts, h) for _, i, p, parts in entries for h in range(hkv)]
    blocks = [[] for _ in range(min(sms, len(items)))]
    for v, item in enumerate(items):
        k, at = divmod(v, len(blocks))
        blocks[len(blocks) - 1 - at if k & 1 else at].append(item)
    return blocks


def parts_before_another_head(sq, sk, heads, hkv, window=0):
    """Parts of split key tiles behind which their block takes an item of another kv head."""
    return sum(x[2] > 1 and x[3] != y[3] for b in key_items(sq, sk, heads, hkv, window) for x, y in zip(b, b[1:]))


# (queries, keys, heads, kv heads, head_dim, window, buckets, max_distance): each has split key tiles, several kv heads and more items than SMs.
SPLIT = {
    "2048": ([2048], [2048], 32, 8, 128, 0, 32, 128),
    "2048 no bias": ([2048], [2048], 32, 8, 64, 0, 0, 0),
    "2048 window": ([2048], [2048], 32, 8, 128, 700, 0, 0),
    "4096 four kv heads": ([4096], [4096], 32, 4, 64, 0, 32, 128),
    "4096 no bias": ([4096], [4096], 32, 8, 128, 0, 0, 0),
    "three": ([2048, 700, 300], [2048, 700, 300], 32, 8, 128, 0, 0, 0),
    "three with a bias": ([2048, 700, 300], [2048, 700, 300], 32, 8, 64, 0, 16, 500),
    "context and window": ([1500, 0, 129], [2100, 77, 129], 24, 6, 64, 1100, 8, 300),
    "more queries than keys": ([2100, 40], [1900, 0], 40, 10, 128, 0, 32, 128),
    "two kv heads": ([3000, 1100], [3000, 1100], 16, 2, 64, 0, 0, 0),
}
