"""Packed attention and the relative position bias at their edges: a maximum of zero, NaN, very low biases, autograd, and a paged cache
whose other rows are NaN.  Bounds are those of test_gpu_relative.py."""
import numpy as np
import pytest
import torch

import paged_kv_attention_03_gb300 as pa
from _packed import values

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(autouse=True)
def _library(cuda):
    pa.pa_read_device_error(clear=True)


def dev(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).cuda()


class Call:
    def __init__(self, sq, sk, heads, hkv, dim, buckets=0, distance=0, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.cu_q, self.cu_k = (np.concatenate([[0], np.cumsum(n)]) for n in (sq, sk))
        self.q, self.dout = normal(sum(sq), heads, dim), normal(sum(sq), heads, dim)
        self.k, self.v = normal(sum(sk), hkv, dim), normal(sum(sk), hkv, dim)
        self.bias = torch.randn(buckets, heads, generator=g, device="cuda") if buckets else None
        self.max_q, self.max_k, self.distance, self.scale = max(sq), max(sk), distance, dim ** -0.5

    def args(self):
        return dev(self.cu_q), dev(self.cu_k), self.max_q, self.max_k, self.scale

    def forward(self, **kw):
        return pa.pa_varlen_attn(self.q, self.k, self.v, *self.args(), bias=self.bias, max_distance=self.distance, **kw)

    def backward(self, out, lse, **kw):
        return pa.pa_varlen_attn_backward(self.dout, self.q, self.k, self.v, out, lse, *self.args(), bias=self.bias,
                                          max_distance=self.distance, **kw)

    def values(self, dout=None):
        return values(self.q, self.k, self.v, self.cu_q, self.cu_k, 0, self.scale, self.bias, self.distance, dout)


@pytest.mark.parametrize("buckets", [0, 16])
def test_rows_beyond_a_maximum_of_zero_are_flagged(buckets):
    c = Call([40, 3], [40, 3], 4, 2, 64, buckets, 64)
    c.max_q = 0
    out, lse = torch.full_like(c.q, 7.0), torch.full(c.q.shape[:2], 7.0, device="cuda")
    c.forward(out=out, lse=lse)
    assert pa.pa_read_device_error() == pa.DEVERR_QUERY_LEN
    assert (out == 7.0).all() and (lse == 7.0).all()
    dq = torch.full_like(c.q, 7.0)
    c.backward(out, lse, dq=dq)
    assert pa.pa_read_device_error() == pa.DEVERR_QUERY_LEN and (dq == 7.0).all()
    c.cu_q = np.array([0, 0, 0])  # no row is in a sequence: nothing is wrong
    c.forward(out=out, lse=lse)
    assert pa.pa_read_device_error() == 0 and (out == 7.0).all()


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("buckets", [0, 16])
def test_a_nan_query_is_no_row_without_keys(dim, buckets):
    c = Call([50, 200], [50, 260], 4, 2, dim, buckets, 64)
    c.q[7, 1] = float("nan")
    c.q[90, 3] = float("nan")
    out, lse = c.forward()
    bad = torch.zeros(c.q.shape[:2], dtype=torch.bool, device="cuda")
    bad[7, 1] = bad[90, 3] = True
    assert torch.equal(lse.isnan(), bad) and torch.equal(out.isnan().all(-1), bad) and torch.equal(out.isnan().any(-1), bad)
    dq = c.backward(out, lse)[0]
    assert dq[7, 1].isnan().all() and dq[90, 3].isnan().all()
    assert pa.pa_read_device_error() == 0
