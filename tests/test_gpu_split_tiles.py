"""dK and dV of key tiles that several blocks share, with several kv heads and blocks that have a next item of another one:
against 64 bits, and bit for bit over repeats and graph replays into gradients full of a sentinel.

Tolerances, with u = 2^-8 and e = 2^-22 (n + 64 + 128 S) (n keys a row, S the largest sum of a logit's absolute terms; a weight
is off by a factor 1 + e at most): (u + 2 e) times the sums of |dS| (dv: of P) for the rounding of an operand and e's use in P twice,
2 e times those of P (N + sum P N), u |result| for the last rounding, and 2^-24 m times the sums for adding m rows up in fp32, in
parts or not.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_03_gb300 as pa
from _packed import SPLIT, values

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(autouse=True)
def _library(cuda):
    pa.pa_read_device_error(clear=True)


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


def within(got, want, tol, what):
    off = (got.double() - want).abs() - tol - 2.0 ** -96
    assert torch.isfinite(got).all(), what
    assert float(off.max()) <= 0.0, f"{what}: {float(off.max())} beyond the bound"


@pytest.mark.parametrize("name", SPLIT)
def test_split_tiles_of_several_kv_heads(name):
    sq, sk, heads, hkv, dim, window, buckets, distance = SPLIT[name]
    g = torch.Generator(device="cuda").manual_seed(len(name))
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    cu_q, cu_k = np.concatenate([[0], np.cumsum(sq)]), np.concatenate([[0], np.cumsum(sk)])
    q, dout = normal(sum(sq), heads, dim), normal(sum(sq), heads, dim)
    k, v = normal(sum(sk), hkv, dim), normal(sum(sk), hkv, dim)
    bias = torch.randn(buckets, heads, generator=g, device="cuda") if buckets else None
    scale = dim ** -0.5
    args = (dev(cu_q), dev(cu_k), max(sq), max(sk), scale, window)
    kw = dict(bias=bias, max_distance=distance)
    out, lse = pa.pa_varlen_attn(q, k, v, *args, **kw)

    def sentinels():
        return dict(dq=torch.full_like(q, 7.0), dk=torch.full_like(k, 7.0), dv=torch.full_like(v, 7.0))

    grads = pa.pa_varlen_attn_backward(dout, q, k, v, out, lse, *args, **kw, **sentinels())
    for _ in range(3):
        for a, b in zip(grads, pa.pa_varlen_attn_backward(dout, q, k, v, out, lse, *args, **kw, **sentinels())):
            assert (a is None and b is None) or torch.equal(a, b)
    again = sentinels()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = pa.pa_varlen_attn_backward(dout, q, k, v, out, lse, *args, **kw, **again)
    for _ in range(3):
        for x in again.values():
            x.fill_(7.0)
        graph.replay()
        for a, b in zip(grads, got):
            assert (a is None and b is None) or torch.equal(a, b)
    assert pa.pa_read_device_error() == 0

    r = values(q, k, v, cu_q, cu_k, window, scale, bias, distance, dout)
    e = 2.0 ** -22 * (max(sk) + 64 + 128 * float(r["logit"].max()))
    sums = 2.0 ** -24 * max(sq) * (heads // hkv)
    dq, dk, dv, dbias = grads
    within(dk, r["dk"], (U + 2 * e + sums) * r["dk_abs"] + 2 * e * r["dk_terms"] + U * r["dk"].abs(), "dk")
    within(dv, r["dv"], (U + 2 * e + sums) * r["dv_abs"] + U * r["dv"].abs(), "dv")
    if buckets:
        within(dbias, r["dbias"], 2 * e * r["dbias_terms"], "dbias")
