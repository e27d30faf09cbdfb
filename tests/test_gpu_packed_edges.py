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


def _paged(c, block, behind_the_ends=0.0, seed=0):
    """The case's keys in shuffled blocks.  Every other row of the cache is NaN, but those behind the end of a sequence in its last
    block, which are read with weight 0."""
    lens = np.diff(c.cu_k)
    blocks = -(-lens // block)
    total = int(blocks.sum()) + 5
    order = np.random.default_rng(seed).permutation(total)
    table = np.full((len(lens), max(int(blocks.max()), 1)), -1)
    hkv, d = c.k.shape[1:]
    caches = [torch.full((total, block, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for i, n in enumerate(lens):
        table[i, :blocks[i]], order = order[:blocks[i]], order[blocks[i]:]
        for cache, rows in zip(caches, (c.k, c.v)):
            for b in range(blocks[i]):
                part = rows[c.cu_k[i] + b * block:min(c.cu_k[i] + (b + 1) * block, c.cu_k[i + 1])]
                cache[table[i, b], :len(part)] = part
                cache[table[i, b], len(part):] = behind_the_ends
    assert sum(int(x.isnan().all(dim=3).all(dim=2).all(dim=1).sum()) for x in caches) == 10
    return *caches, dev(table), dev(lens)


@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("heads,hkv,dim", [(8, 2, 64), (20, 1, 128)])
def test_blocks_of_nobody_are_not_read(heads, hkv, dim, block):
    new, lens = [70, 1, 33, 1], [70, 600, 300, 17]
    c = Call(new, lens, heads, hkv, dim, 32, 128)
    k, v, table, seq_lens = _paged(c, block)
    r = c.values()
    e = 2.0 ** -22 * (600 + 64 + 128 * float(r["logit"].max()))
    tol = (U + 2 * e) * r["out_abs"] + 2 * U * r["out"].abs()
    out = pa.pa_varlen_prefill_bias(c.q, k, v, dev(c.cu_q), seq_lens, table, 70, 600, c.scale, c.bias, 128)
    assert torch.isfinite(out).all() and ((out.double() - r["out"]).abs() <= tol).all()
    last = torch.as_tensor(c.cu_q[1:] - 1).cuda()
    for splits in (0, 1, 4):
        out = pa.pa_decode_bias(c.q[last], k, v, table, seq_lens, 600, c.scale, c.bias, 128, 0, splits)
        assert torch.isfinite(out).all() and ((out.double() - r["out"][last]).abs() <= tol[last]).all()
    assert pa.pa_read_device_error() == 0


@pytest.mark.parametrize("splits", [0, 1, 3])
def test_decode_keeps_nan(splits):
    """A NaN query, key or bias gives NaN with the bias as without it, however the keys are split."""
    lens = [40, 300, 90]
    c = Call([1, 1, 1], lens, 4, 2, 64, 16, 64)
    k, v, table, seq_lens = _paged(c, 16)
    c.q[0, 2] = float("nan")
    k[table[2, 1], 3, 1] = float("nan")
    c.bias[5, 0] = float("nan")
    out = pa.pa_decode_bias(c.q, k, v, table, seq_lens, 300, c.scale, c.bias, 64, 0, splits)
    nan = out.isnan().all(-1)
    want = torch.zeros(3, 4, dtype=torch.bool, device="cuda")
    want[0, 2] = want[2, 2] = want[2, 3] = True
    want[:, 0] = True  # distance 5 is in every sequence
    assert torch.equal(nan, want) and torch.equal(out.isnan().any(-1), want)


@pytest.mark.parametrize("low", [-1e9, -3e7])
@pytest.mark.parametrize("heads,hkv,dim", [(4, 2, 64), (8, 1, 128)])
def test_rows_of_nothing_but_very_low_biases_have_no_gradient(low, heads, hkv, dim):
    """lse of such rows has no digits left for e^(s - lse).  Keys with such a bias beside others have weight 0."""
    c = Call([200, 1, 30], [260, 1, 30], heads, hkv, dim, 16, 64)
    c.bias[0, 1] = low  # a position does not see itself: the first one of a sequence sees nothing else
    c.bias[:, 3] = low
    c.bias[9:, 2] = low
    out, lse = c.forward()
    grads = c.backward(out, lse)
    assert pa.pa_read_device_error() == 0
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    dout = c.dout.clone()
    dout[lse < -1e6] = 0.0
    assert (dout[:, 3] == 0).all() and (dout[200, 1] == 0).all() and (dout[:, 0] == c.dout[:, 0]).all()
    c.bias[c.bias == low] = float("-inf")
    r = c.values(dout)
    e = 2.0 ** -22 * (260 + 64 + 128 * float(r["logit"].max()))
    moved = U * r["ds_abs"] + 2 * e * r["mean"]
    tols = {"dq": (U + 2 * e) * r["dq_abs"] + 2 * e * r["dq_terms"] + moved[..., None] * r["dq_rows"], "dk": (U + 2 * e) * r["dk_abs"] + 2 * e * r["dk_terms"],
            "dv": (U + 2 * e) * r["dv_abs"], "dbias": 2 * e * r["dbias_terms"]}
    for name, got in zip(("dq", "dk", "dv", "dbias"), grads):
        assert torch.isfinite(got).all(), name
        assert ((got.double() - r[name]).abs() <= tols[name] + U * r[name].abs() + 2.0 ** -96).all(), name


def test_a_call_that_records_no_graph_says_so():
    import warnings
    c = Call([20], [20], 4, 2, 64, 16, 64)
    for name in ("q", "k", "v", "bias"):
        t = getattr(c, name)
        t.requires_grad_(True)
        with pytest.warns(RuntimeWarning, match="pa_varlen_attn_backward"):
            out, lse = c.forward()
        assert not out.requires_grad and not lse.requires_grad
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            with torch.no_grad():
                c.forward()
            t.requires_grad_(False)
            c.forward()


def test_an_autograd_function_of_the_two_calls():
    """What a model wraps the two calls in: no warning, and the gradients of the calls."""
    import warnings
    c = Call([70, 130], [70, 130], 4, 2, 64, 16, 64)

    class Attention(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, v, bias):
            c.q, c.k, c.v, c.bias = q, k, v, bias
            out, lse = c.forward()
            ctx.save_for_backward(q, k, v, bias, out, lse)
            return out

        @staticmethod
        def backward(ctx, dout):
            q, k, v, bias, out, lse = ctx.saved_tensors
            return pa.pa_varlen_attn_backward(dout.contiguous(), q, k, v, out, lse, *c.args(), bias=bias, max_distance=64)

    out, lse = c.forward()
    want = c.backward(out, lse)
    leaves = [t.clone().requires_grad_(True) for t in (c.q, c.k, c.v, c.bias)]
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        Attention.apply(*leaves).backward(c.dout)
    for t, g in zip(leaves, want):
        assert torch.equal(t.grad, g)
