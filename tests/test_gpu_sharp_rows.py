"""dq of rows whose weight lies on few of many keys: their dS nearly cancel, so what stands for sum_j P_j dP_j has to be far more
exact than dout . out with a rounded out.

Tolerance, with u = 2^-8: dS is rounded to bf16 and so is dq (u on each); the sum over the keys is known to u sum_j |dS_j|, which
moves dq by that times scale sum P |k|.  Logits are sums of 8 products of 16 terms in fp32, off by d = 2^-20 S (S the largest sum
of their absolute terms), so dS by 3 d of itself; and a row's weights are all off by one factor 1 + n, n = 2^-22 (4 + |lse|)
(lse and its product with log2 e are rounded), or each by d: that moves the sum by (d + n) sum P N.
"""
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


def step(sharp, sq, sk, heads, hkv, dim, window=0, buckets=0, distance=0, seed=0):
    """Inputs whose logits are `sharp` times those of normal ones, outputs and gradients, and their 64-bit values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    cu_q, cu_k = np.concatenate([[0], np.cumsum(sq)]), np.concatenate([[0], np.cumsum(sk)])
    q, dout = (normal(sum(sq), heads, dim) * sharp).bfloat16(), normal(sum(sq), heads, dim).bfloat16()
    k, v = normal(sum(sk), hkv, dim).bfloat16(), normal(sum(sk), hkv, dim).bfloat16()
    bias = normal(buckets, heads) if buckets else None
    args = (dev(cu_q), dev(cu_k), max(sq), max(sk), dim ** -0.5, window)
    kw = dict(bias=bias, max_distance=distance)
    out, lse = pa.pa_varlen_attn(q, k, v, *args, **kw)
    grads = pa.pa_varlen_attn_backward(dout, q, k, v, out, lse, *args, **kw)
    for a, b in zip(grads, pa.pa_varlen_attn_backward(dout, q, k, v, out, lse, *args, **kw)):
        assert (a is None and b is None) or torch.equal(a, b)
    assert pa.pa_read_device_error() == 0
    return grads, values(q, k, v, cu_q, cu_k, window, dim ** -0.5, bias, distance, dout)


def check_dq(dq, r):
    d = 2.0 ** -20 * float(r["logit"].max())
    n = 2.0 ** -22 * (4 + r["lse"].abs().nan_to_num(posinf=0.0))
    moved = (U * r["ds_abs"] + (d + n) * r["mean"])[..., None] * r["dq_rows"]
    tol = (U + 3 * d) * r["dq_abs"] + moved + U * r["dq"].abs() + 2.0 ** -96
    assert torch.isfinite(dq).all()
    beyond = ((dq.double() - r["dq"]).abs() / tol).flatten(2).amax(2)
    assert float(beyond.max()) <= 1.0, f"{int((beyond > 1).sum())} of {beyond.numel()} rows beyond the bound, by up to {float(beyond.max()):.3g}"


@pytest.mark.parametrize("sharp", [1, 4, 8, 30])
@pytest.mark.parametrize("heads,hkv,dim", [(4, 2, 128), (3, 3, 64)])
@pytest.mark.parametrize("window,buckets,distance", [(0, 0, 0), (200, 0, 0), (0, 32, 128), (0, 8, 20), (300, 16, 100)])
def test_dq_of_sharp_rows(sharp, heads, hkv, dim, window, buckets, distance):
    (dq, _, _, _), r = step(sharp, [512, 90, 300], [512, 90, 700], heads, hkv, dim, window, buckets, distance, seed=sharp)
    check_dq(dq, r)


@pytest.mark.parametrize("buckets,distance", [(0, 0), (32, 128)])
def test_many_sharp_items_a_block(buckets, distance):
    """Several items for each of the GPU's blocks, sharp ones and others, of one step and of several."""
    sq = [130, 1, 700, 128, 257, 64, 300] * 6
    (dq, _, _, _), r = step(6, sq, [n + 150 for n in sq], 16, 4, 64, 0, buckets, distance)
    check_dq(dq, r)
