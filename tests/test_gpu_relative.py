"""Packed attention, its gradient and the learned relative position bias on the GPU, against the fp64 oracle.

Tolerances, with u = 2^-8 (half a step of bf16, relative):
 * logits are fp32 sums of at most 128 products and a bias, so a weight is off by at most a factor 1 + e,
   e = 2^-22 (n + 64 + 128 S), n keys a row and S the largest sum of a logit's absolute terms (the sums of
   e^s and their use, twice, in the exponent);
 * out: weights are rounded to bf16 and so is the result: (u + e) sum P |v| + u |out|, taken twice for e's use in
   the numerator and the denominator: (u + 2 e);
 * lse: 2^-23 (n + 64 + 128 S);
 * dv: (u + 2 e) sum P |dout| + u |dv|;
 * dq, dk: dS is rounded to bf16 (u |dS|) and off by 2 e (|dS| + P (N + M)) (the names of the oracle); dQ starts from
   dout . out with a rounded out, which moves a row's dS by P |dout| . tol(out);
 * dbias: no rounding: 2 e (|dS| + P (N + M));
 * weights below 2^-126 are flushed to zero: at most 2^20 terms of at most 2^10 times that each, 2^-96.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_03_gb300 as pa
from oracle import relative

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


@pytest.fixture(autouse=True)
def _library(cuda):
    pa.pa_read_device_error(clear=True)


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


class Case:
    def __init__(self, sq, sk, heads, hkv, dim, window=0, buckets=0, distance=0, seed=0, behind=0, bias_scale=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
        self.cu_q, self.cu_k = offsets(sq), offsets(sk)
        self.max_q, self.max_k, self.window, self.distance = max(sq, default=0), max(sk, default=0), window, distance
        self.q, self.dout = (normal(int(self.cu_q[-1]) + behind, heads, dim) for _ in range(2))
        self.k, self.v = (normal(int(self.cu_k[-1]) + behind, hkv, dim) for _ in range(2))
        self.bias = bias_scale * torch.randn(buckets, heads, generator=g, device="cuda") if buckets else None
        self.scale = dim ** -0.5

    def forward(self, **kw):
        return pa.pa_varlen_attn(self.q, self.k, self.v, dev(self.cu_q), dev(self.cu_k), self.max_q, self.max_k, self.scale, self.window,
                                 bias=self.bias, max_distance=self.distance, **kw)

    def backward(self, out, lse, **kw):
        return pa.pa_varlen_attn_backward(self.dout, self.q, self.k, self.v, out, lse, dev(self.cu_q), dev(self.cu_k), self.max_q, self.max_k,
                                          self.scale, self.window, bias=self.bias, max_distance=self.distance, **kw)

    def oracle(self, grad=True):
        return relative.attention(f64(self.q), f64(self.k), f64(self.v), self.cu_q, self.cu_k, self.window, self.scale,
                                  None if self.bias is None else f64(self.bias), self.distance, f64(self.dout) if grad else None)


def within(got, want, tol, what):
    got = f64(got)
    fine = np.isfinite(want)
    np.testing.assert_array_equal(np.where(fine, 0.0, want), np.where(fine, 0.0, np.where(np.isnan(want), np.nan, got)), err_msg=what)
    off = np.abs(got[fine] - want[fine]) - tol[fine] - 2.0 ** -96
    assert not np.isnan(off).any() and off.max(initial=-1.0) <= 0.0, f"{what}: {off.max()} beyond the bound"


def check(c, out, lse, grads=None):
    r = c.oracle(grads is not None)
    assert pa.pa_read_device_error() == 0
    keys = max(c.max_k, 1)
    e = 2.0 ** -22 * (keys + 64 + 128 * float(np.max(r["logit"], initial=0.0)))
    tol_out = (U + 2 * e) * r["out_abs"] + U * np.abs(r["out"])
    within(out, r["out"], tol_out, "out")
    within(lse, r["lse"], np.full(r["lse"].shape, e / 2), "lse")
    if grads is None:
        return
    dq, dk, dv, dbias = grads
    moved = (np.abs(f64(c.dout)) * np.nan_to_num(tol_out)).sum(-1, keepdims=True)
    within(dv, r["dv"], (U + 2 * e) * r["dv_abs"] + U * np.abs(r["dv"]), "dv")
    within(dq, r["dq"], (U + 2 * e) * r["dq_abs"] + 2 * e * r["dq_terms"] + moved * r["dq_rows"] * (1 + U) + U * np.abs(r["dq"]), "dq")
    within(dk, r["dk"], (U + 2 * e) * r["dk_abs"] + 2 * e * r["dk_terms"] + U * np.abs(r["dk"]), "dk")
    if c.bias is not None:
        within(dbias, r["dbias"], 2 * e * r["dbias_terms"], "dbias")
    else:
        assert dbias is None


def both(c):
    out, lse = c.forward()
    return out, lse, c.backward(out, lse)


LENGTHS = {
    "one": ([1], [1]),
    "short": ([5, 1, 31], [5, 1, 31]),
    "tiles": ([127, 128, 129], [127, 128, 129]),
    "ragged": ([300, 17, 0, 255], [300, 17, 0, 255]),
    "context": ([1, 40, 130, 7], [200, 90, 390, 7]),
    "empty rows": ([200, 3, 130, 5], [60, 0, 129, 3]),
    "no queries": ([0, 64, 0], [33, 64, 140]),
    "long": ([700], [1100]),
}


@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("heads,hkv,dim", [(2, 2, 64), (8, 2, 128), (5, 1, 64), (14, 2, 128)])
@pytest.mark.parametrize("window,buckets,distance", [(0, 0, 0), (0, 32, 128), (37, 0, 0), (150, 8, 300), (0, 6, 4)])
def test_packed_and_gradient(lengths, heads, hkv, dim, window, buckets, distance):
    c = Case(*LENGTHS[lengths], heads, hkv, dim, window, buckets, distance, seed=len(lengths))
    out, lse, grads = both(c)
    check(c, out, lse, grads)


@pytest.mark.parametrize("heads,hkv,dim", [(12, 12, 64), (16, 4, 128)])
@pytest.mark.parametrize("window,buckets,distance", [(0, 32, 128), (0, 0, 0), (0, 16, 30000), (40, 8, 20), (200, 32, 128)])
def test_many_tiles_a_block(heads, hkv, dim, window, buckets, distance):
    """Several items for each of the GPU's persistent blocks, of one tile and of several, empty ones among them."""
    g = np.random.default_rng(4)
    sq = g.integers(0, 200, 90).tolist() + [400, 129]
    sk = [n + int(m) for n, m in zip(sq, g.integers(-30, 90, 92))]
    c = Case(sq, [max(n, 0) for n in sk], heads, hkv, dim, window, buckets, distance, seed=6)
    out, lse, grads = both(c)
    check(c, out, lse, grads)
    for a, b in zip((out, lse, *grads), (lambda r: (r[0], r[1], *r[2]))(both(c))):
        assert (a is None and b is None) or torch.equal(a, b)


def test_thousands_of_short_sequences():
    """More sequences than the list's block takes in one round; most of them empty or of a token or two."""
    g = np.random.default_rng(8)
    sq = g.integers(0, 4, 5000)
    sk = np.maximum(sq + g.integers(-1, 3, 5000), 0)
    c = Case(sq.tolist(), sk.tolist(), 2, 1, 64, 0, 8, 9)
    out, lse, grads = both(c)
    check(c, out, lse, grads)


def test_rows_far_apart():
    """Rows of q, k, v and of the gradients so far apart that offsets pass 2^32 bytes and 2^31 elements."""
    heads, hkv, d, step = 4, 2, 64, 1 << 23
    c = Case([200, 77], [200, 77], heads, hkv, d, 0, 32, 128)
    out, lse, grads = both(c)
    base = torch.empty(277 * step, dtype=torch.bfloat16, device="cuda").view(277, step)
    split = lambda t: (t[:, : heads * d].view(-1, heads, d), t[:, heads * d:(heads + hkv) * d].view(-1, hkv, d),  # noqa: E731
                       t[:, (heads + hkv) * d:(heads + 2 * hkv) * d].view(-1, hkv, d))
    wide = split(base)
    for mine, theirs in zip(wide, (c.q, c.k, c.v)):
        mine.copy_(theirs)
    c.q, c.k, c.v = wide
    out2, lse2 = c.forward()
    dq, dk, dv = split(base[:, step // 2:])
    grads2 = c.backward(out2, lse2, dq=dq, dk=dk, dv=dv)
    for a, b in zip((out, lse, *grads), (out2, lse2, *grads2)):
        assert torch.equal(a, b)


def test_sequences_that_begin_behind_row_0():
    """Rows before the first sequence are left as they were too."""
    c = Case([50, 90], [70, 90], 4, 2, 64, 0, 16, 64)
    want = both(c)
    pad = lambda t: torch.cat([torch.full_like(t[:13], float("nan")), t])  # noqa: E731
    moved = Case([50, 90], [70, 90], 4, 2, 64, 0, 16, 64)
    moved.q, moved.k, moved.v, moved.dout = pad(c.q), pad(c.k), pad(c.v), pad(c.dout)
    moved.cu_q, moved.cu_k = c.cu_q + 13, c.cu_k + 13
    fill = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    out, lse = moved.forward(out=fill(moved.q), lse=torch.full(moved.q.shape[:2], 7.0, device="cuda"))
    dq, dk, dv, dbias = moved.backward(out, lse, dq=fill(moved.q), dk=fill(moved.k), dv=fill(moved.v))
    for got, ref in zip((out, lse, dq, dk, dv), (want[0], want[1], *want[2])):
        assert (got[:13] == 7.0).all() and torch.equal(got[13:], ref)
    assert torch.equal(dbias, want[2][3])


@pytest.mark.parametrize("heads,hkv", [(64, 1), (32, 2), (33, 1), (3, 3), (128, 2)])
def test_head_layouts(heads, hkv):
    c = Case([70, 9], [70, 30], heads, hkv, 128, 0, 32, 128)
    out, lse, grads = both(c)
    check(c, out, lse, grads)


@pytest.mark.parametrize("buckets,distance", [(2, 2), (128, 32768), (127, 64), (64, 700), (32, 17)])
def test_bucket_counts(buckets, distance):
    c = Case([600, 64], [900, 64], 4, 2, 64, 0, buckets, distance, seed=buckets)
    out, lse, grads = both(c)
    check(c, out, lse, grads)
    first = relative.first_distances(buckets, distance) + [1 << 30]
    for b in range(buckets):  # buckets that no pair reaches have no gradient at all
        if first[b] > 899 or first[b] == first[b + 1]:
            assert (grads[3][b] == 0).all(), b


def test_a_window_before_the_last_bucket_leaves_it_at_zero():
    c = Case([300], [300], 4, 2, 64, 113, 32, 128)
    assert relative.first_distances(32, 128)[-1] == 113
    out, lse, grads = both(c)
    check(c, out, lse, grads)
    assert (grads[3][-1] == 0).all()
    c = Case([300], [300], 4, 2, 64, 114, 32, 128)
    out, lse, grads = both(c)
    check(c, out, lse, grads)
    assert (grads[3][-1] != 0).all()


def test_the_bias_gradient_keeps_fp32():
    """Errors of dbias' terms are those of fp32 (about 1e-6 of a term, random): 1e-5 of its norm.  With dS rounded to bf16, or sums of
    dout . out for a rounded out, they would be about 1e-4."""
    c = Case([1500, 400], [1500, 400], 4, 2, 128, 0, 32, 128)
    _, _, grads = both(c)
    want = c.oracle()["dbias"]
    assert np.linalg.norm(f64(grads[3]) - want) <= 1e-5 * np.linalg.norm(want)


@pytest.mark.parametrize("how", ["minus infinity", "lowest", "large", "large and far", "all hidden"])
def test_bias_values(how):
    c = Case([200, 30], [260, 30], 4, 2, 64, 0, 16, 64)
    if how == "large":
        c.bias *= 40.0
    elif how == "large and far":  # the last bucket's far beyond the others'
        c.bias[-1] = torch.tensor([-9000.0, 700.0, -65.0, 63.0])
    elif how == "all hidden":
        c.bias[:, 1] = float("-inf")
        c.bias[0, 2] = float("-inf")
    else:
        c.bias[::3] = float("-inf") if how == "minus infinity" else torch.finfo(torch.float32).min
    out, lse, grads = both(c)
    if how == "lowest":  # hides keys as -inf does
        hidden = Case([200, 30], [260, 30], 4, 2, 64, 0, 16, 64)
        hidden.bias[::3] = float("-inf")
        for a, b in zip((out, lse, *grads), (lambda r: (r[0], r[1], *r[2]))(both(hidden))):
            assert torch.equal(a, b)
        return
    if how == "all hidden":
        assert (out[:, 1] == 0).all() and torch.isneginf(lse[:, 1]).all()
        assert (grads[0][:, 1] == 0).all() and (grads[3][:, 1] == 0).all()
    check(c, out, lse, grads)


def test_slices_of_one_projection():
    """q, k, v and the gradients as slices of [T, (H + 2 Hkv) D] rows: the same bits as contiguous ones, and nothing beside them."""
    heads, hkv, d = 8, 2, 128
    c = Case([130, 77], [130, 77], heads, hkv, d, 0, 32, 128)
    out, lse, grads = both(c)
    row = torch.full((207, (heads + 2 * hkv) * d + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    split = lambda t: (t[:, : heads * d].view(-1, heads, d), t[:, heads * d:(heads + hkv) * d].view(-1, hkv, d),  # noqa: E731
                       t[:, (heads + hkv) * d:(heads + 2 * hkv) * d].view(-1, hkv, d))
    q, k, v = split(row)
    q.copy_(c.q), k.copy_(c.k), v.copy_(c.v)
    c.q, c.k, c.v = q, k, v
    out2, lse2 = c.forward()
    grad_row = torch.full_like(row, 5.0)
    dq, dk, dv = split(grad_row)
    grads2 = c.backward(out2, lse2, dq=dq, dk=dk, dv=dv)
    for a, b in zip((out, lse, *grads), (out2, lse2, *grads2)):
        assert torch.equal(a, b)
    assert (grad_row[:, -8:] == 5.0).all() and (row[:, -8:] == 3.0).all()


def test_rows_behind_the_last_sequence_and_what_stands_beside_a_sequence():
    """NaN in another sequence and behind the last one reaches nobody; rows behind are left as they were."""
    c = Case([100, 20, 33], [150, 40, 33], 4, 2, 64, 0, 32, 128, behind=9)
    want = c.oracle()
    for t, cu in ((c.q, c.cu_q), (c.dout, c.cu_q), (c.k, c.cu_k), (c.v, c.cu_k)):
        t[cu[1]:cu[2]] = float("nan")
        t[cu[-1]:] = float("nan")
    fill = lambda t: torch.full_like(t, 7.0)  # noqa: E731
    out, lse = c.forward(out=fill(c.q), lse=torch.full(c.q.shape[:2], 7.0, device="cuda"))
    dq, dk, dv, _ = c.backward(out, lse, dq=fill(c.q), dk=fill(c.k), dv=fill(c.v))
    for got, name, cu in ((out, "out", c.cu_q), (lse, "lse", c.cu_q), (dq, "dq", c.cu_q), (dk, "dk", c.cu_k), (dv, "dv", c.cu_k)):
        assert (got[cu[-1]:] == 7.0).all(), name
        for a, b in ((cu[0], cu[1]), (cu[2], cu[3])):
            assert torch.isfinite(got[a:b]).all(), name
            assert np.abs(f64(got[a:b]) - want[name][a:b]).max() < 0.1, name  # (bounds are the other tests')


@pytest.mark.parametrize("heads,hkv,dim", [(16, 1, 64), (16, 1, 128), (27, 3, 128), (9, 1, 64)])
@pytest.mark.parametrize("window,buckets,distance", [(0, 0, 0), (0, 32, 128), (333, 16, 500)])
def test_few_kv_heads_of_many_queries(heads, hkv, dim, window, buckets, distance):
    """Key tiles of many steps, which several blocks share: sums in parts, the same bits every time."""
    c = Case([901, 0, 40, 128, 1], [901, 20, 300, 128, 700], heads, hkv, dim, window, buckets, distance, seed=8)
    out, lse, grads = both(c)
    check(c, out, lse, grads)
    again = [torch.full_like(x, 7.0) for x in grads if x is not None]
    kw = dict(zip(("dq", "dk", "dv", "dbias"), again))
    graph = torch.cuda.CUDAGraph()
    cu_q, cu_k = dev(c.cu_q), dev(c.cu_k)
    with torch.cuda.graph(graph):
        pa.pa_varlen_attn_backward(c.dout, c.q, c.k, c.v, out, lse, cu_q, cu_k, c.max_q, c.max_k, c.scale, c.window, bias=c.bias,
                                   max_distance=c.distance, **kw)
    for _ in range(3):
        for x in again:
            x.fill_(7.0)
        graph.replay()
        for x, y in zip(again, grads):
            assert torch.equal(x, y)
    assert pa.pa_read_device_error() == 0


def test_bad_offsets_are_flagged_and_left_out():
    c = Case([40, 40, 40], [40, 40, 40], 4, 2, 64, 0, 32, 128)
    good = both(c)
    cu_q, cu_k = c.cu_q.copy(), c.cu_k.copy()
    for which, bad, flag in ((0, [0, 40, 80, 121], pa.DEVERR_QUERY_LEN), (0, [0, 40, 30, 70], pa.DEVERR_QUERY_LEN),
                             (1, [0, 40, 80, 130], pa.DEVERR_SEQ_RANGE), (1, [-5, 35, 75, 115], pa.DEVERR_SEQ_RANGE)):
        c.cu_q, c.cu_k = (np.array(bad) if which == 0 else cu_q), (np.array(bad) if which == 1 else cu_k)
        c.max_q = c.max_k = 50
        out = torch.full_like(c.q, 7.0)
        lse = good[1].clone()
        c.forward(out=out, lse=lse)
        assert pa.pa_read_device_error() & flag
        c.backward(out, lse)
        assert pa.pa_read_device_error() & flag
    c.cu_q, c.cu_k = cu_q, cu_k
    c.max_q = 39  # shorter than the sequences
    out.fill_(7.0)
    c.forward(out=out)
    assert pa.pa_read_device_error() & pa.DEVERR_QUERY_LEN and (out == 7.0).all()
    c.max_q = 50
    again = both(c)
    assert pa.pa_read_device_error() == 0
    for a, b in zip((good[0], good[1], *good[2]), (again[0], again[1], *again[2])):
        assert torch.equal(a, b)


def test_offsets_that_go_back_and_forth():
    """Sequences over the same rows, between others of negative length, have more tiles than the rows have."""
    c = Case([1000], [1000], 4, 2, 64, 0, 32, 128)
    good = both(c)
    back = [0] + [1000, 0] * 40
    fill = lambda x: torch.full_like(x, 7.0)  # noqa: E731
    cu_q, cu_k = c.cu_q, c.cu_k
    for cu in ((back, back), (back, [0] + [30, 60] * 40), ([0] + [30, 60] * 40, back)):
        c.cu_q, c.cu_k = np.array(cu[0]), np.array(cu[1])
        dq, dk, dv, dbias = c.backward(good[0], good[1], dq=fill(c.q), dk=fill(c.k), dv=fill(c.v))
        assert pa.pa_read_device_error() & (pa.DEVERR_QUERY_LEN | pa.DEVERR_SEQ_RANGE)
        if cu[0] is back and cu[1] is back:
            assert (dq == 7.0).all() and (dk == 7.0).all() and (dv == 7.0).all() and (dbias == 0).all()
    c.cu_q, c.cu_k = cu_q, cu_k
    again = both(c)
    assert pa.pa_read_device_error() == 0
    for a, b in zip((good[0], good[1], *good[2]), (again[0], again[1], *again[2])):
        assert torch.equal(a, b)


def test_nothing_to_do():
    for sq, sk in (([], []), ([0, 0], [0, 0]), ([0], [30]), ([30], [0])):
        c = Case(sq, sk, 4, 2, 64, 0, 32, 128)
        if not sq:
            c.cu_q = c.cu_k = np.zeros(1, np.int64)
        out, lse, (dq, dk, dv, dbias) = both(c)
        assert pa.pa_read_device_error() == 0
        assert (out == 0).all() and torch.isneginf(lse).all() and (dbias == 0).all()
        for t in (dq, dk, dv):
            assert (t == 0).all()


def test_graph_streams_and_repeats():
    """Equal bits eagerly, on a side stream beside another call, and from a replayed graph over new inputs."""
    c = Case([300, 40, 129], [300, 90, 129], 8, 2, 128, 0, 32, 128)
    other = Case([257, 33], [257, 33], 8, 2, 128, 100, 16, 64, seed=5)
    flat = lambda r: (r[0], r[1], *r[2])  # noqa: E731
    want, want_other = flat(both(c)), flat(both(other))
    for a, b in zip(want, flat(both(c))):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            got = flat(both(c))
        with torch.cuda.stream(s2):
            got_other = flat(both(other))
        torch.cuda.synchronize()
        for a, b in zip((*want, *want_other), (*got, *got_other)):
            assert torch.equal(a, b)
    cu_q, cu_k = dev(c.cu_q), dev(c.cu_k)
    outs = [torch.empty_like(t) for t in want]
    ws = torch.empty(pa.pa_varlen_attn_backward_workspace_size(len(c.q), len(c.k), 3, 8, 32, 128), dtype=torch.uint8, device="cuda")

    def step():
        pa.pa_varlen_attn(c.q, c.k, c.v, cu_q, cu_k, 300, 300, c.scale, bias=c.bias, max_distance=128, out=outs[0], lse=outs[1], workspace=ws)
        pa.pa_varlen_attn_backward(c.dout, c.q, c.k, c.v, outs[0], outs[1], cu_q, cu_k, 300, 300, c.scale, bias=c.bias, max_distance=128,
                                   dq=outs[2], dk=outs[3], dv=outs[4], dbias=outs[5], workspace=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for t in outs:
            t.fill_(1.0)
        graph.replay()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)
    # new inputs and other lengths within the declared maximum
    new = Case([300, 40, 129], [300, 90, 129], 8, 2, 128, 0, 32, 128, seed=9)
    new.cu_q, new.cu_k = offsets([100, 240, 129]), offsets([130, 260, 129])
    for mine, theirs in ((c.q, new.q), (c.k, new.k), (c.v, new.v), (c.dout, new.dout), (c.bias, new.bias), (cu_q, dev(new.cu_q)),
                         (cu_k, dev(new.cu_k))):
        mine.copy_(theirs)
    graph.replay()
    for a, b in zip(outs, flat(both(new))):
        assert torch.equal(a, b)


def test_binding_refusals():
    c = Case([20], [20], 4, 2, 64, 0, 16, 64)
    out, lse = c.forward()
    with pytest.raises(TypeError):
        c.forward(out=out.float())
    with pytest.raises(ValueError):
        c.forward(lse=lse[:-1])
    with pytest.raises(ValueError):
        c.backward(out.transpose(0, 1), lse)
    with pytest.raises(ValueError):
        c.backward(out, lse, dk=torch.empty(20, 2, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2))
    with pytest.raises(ValueError):  # one row for all
        c.backward(out, lse, dq=torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda").expand(20, 4, 64))
    with pytest.raises(ValueError):
        c.forward(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(pa.PAError):
        c.forward(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    q = c.q
    for bad in (q.float(), q.cpu()):
        c.q = bad
        with pytest.raises((TypeError, ValueError)):
            c.forward()
    c.q, bias = q, c.bias
    for bad in (bias.double(), bias.T, bias[:, :3], bias[0]):
        c.bias = bad
        with pytest.raises((TypeError, ValueError)):
            c.forward()
    c.bias, c.distance = bias, 8
    with pytest.raises(pa.PAError):
        c.forward()


# ------------------------------------------------------------- over the paged cache ---
class Paged:
    """The keys of a packed case in a paged cache of shuffled blocks; all other rows of the cache are NaN."""

    def __init__(self, c, block, seed=0):
        lens = np.diff(c.cu_k)
        blocks = -(-lens // block)
        self.num_blocks = int(blocks.sum()) + 3
        order = np.random.default_rng(seed).permutation(self.num_blocks)
        self.table = np.full((len(lens), max(int(blocks.max(initial=1)), 1)), -1)
        hkv, d = c.k.shape[1:]
        self.k, self.v = (torch.full((self.num_blocks, block, hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.slots = np.zeros(int(c.cu_k[-1]), np.int64)
        for i, n in enumerate(lens):
            self.table[i, :blocks[i]], order = order[:blocks[i]], order[blocks[i]:]
            j = np.arange(n)
            self.slots[c.cu_k[i]:c.cu_k[i + 1]] = self.table[i, j // block] * block + j % block
        self.lens = lens
        at = torch.as_tensor(self.slots).cuda()
        self.k.view(-1, hkv, d)[at], self.v.view(-1, hkv, d)[at] = c.k[: len(self.slots)], c.v[: len(self.slots)]
        # The block of a sequence's end is read as a whole, keys behind the end with weight 0.
        self.k.nan_to_num_(0.0), self.v.nan_to_num_(0.0)


def paged_tolerance(c, r):
    """As `out` above; the paged kernels' denominators sum the rounded weights, which adds u |out| at most."""
    e = 2.0 ** -22 * (max(c.max_k, 1) + 64 + 128 * float(np.max(r["logit"], initial=0.0)))
    return (U + 2 * e) * r["out_abs"] + 2 * U * np.abs(r["out"])


@pytest.mark.parametrize("heads,hkv,dim,block", [(8, 2, 64, 16), (32, 8, 128, 16), (5, 1, 128, 64), (32, 2, 64, 4), (40, 1, 128, 16)])
@pytest.mark.parametrize("window,buckets,distance", [(0, 32, 128), (0, 64, 2000), (90, 8, 300), (0, 2, 2)])
@pytest.mark.parametrize("splits", [0, 1, 3])
def test_decode(heads, hkv, dim, block, window, buckets, distance, splits):
    lens = [1, 17, 0, 600, 113, 114, 2000]
    c = Case([1 if n else 0 for n in lens], lens, heads, hkv, dim, window, buckets, distance, seed=block)
    p = Paged(c, block)
    q = torch.randn(len(lens), heads, dim, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").bfloat16()
    rows = [i for i, n in enumerate(lens) if n]
    q[rows] = c.q
    out = pa.pa_decode_bias(q, p.k, p.v, dev(p.table), dev(p.lens), 2000, c.scale, c.bias, distance, window, splits)
    assert pa.pa_read_device_error() == 0
    r = c.oracle(False)
    within(out[rows], r["out"], paged_tolerance(c, r), "out")
    assert (out[2] == 0).all()


@pytest.mark.parametrize("heads,hkv,dim,block", [(8, 2, 64, 16), (32, 8, 128, 16), (5, 1, 128, 64), (64, 1, 64, 32)])
@pytest.mark.parametrize("window,buckets,distance", [(0, 32, 128), (0, 64, 2000), (90, 8, 300), (0, 2, 2)])
@pytest.mark.parametrize("given", ["seq_lens", "cu_seqlens_k"])
def test_prefill(heads, hkv, dim, block, window, buckets, distance, given):
    new, lens = [130, 1, 3, 300, 1, 64], [130, 1, 200, 700, 913, 64]
    c = Case(new, lens, heads, hkv, dim, window, buckets, distance, seed=block)
    p = Paged(c, block)
    kw = {"cu_seqlens_k": dev(c.cu_k)} if given == "cu_seqlens_k" else {}
    out = pa.pa_varlen_prefill_bias(c.q, p.k, p.v, dev(c.cu_q), None if kw else dev(p.lens), dev(p.table), 300, 1000, c.scale, c.bias,
                                    distance, window, **kw)
    assert pa.pa_read_device_error() == 0
    r = c.oracle(False)
    within(out, r["out"], paged_tolerance(c, r), "out")


def test_hidden_keys_in_decode_and_prefill():
    """A bias of -inf hides keys, all of them in one head."""
    new, lens = [1, 60], [500, 200]
    c = Case(new, lens, 4, 2, 64, 0, 16, 64)
    c.bias[3:9] = float("-inf")
    c.bias[:, 2] = float("-inf")
    p = Paged(c, 16)
    r = c.oracle(False)
    out = pa.pa_varlen_prefill_bias(c.q, p.k, p.v, dev(c.cu_q), dev(p.lens), dev(p.table), 60, 500, c.scale, c.bias, 64)
    within(out, r["out"], paged_tolerance(c, r), "prefill")
    for splits in (1, 5):
        out = pa.pa_decode_bias(c.q[:1], p.k, p.v, dev(p.table[:1]), dev(p.lens[:1]), 500, c.scale, c.bias, 64, 0, splits)
        within(out, r["out"][:1], paged_tolerance(c, r)[:1], "decode")


def test_a_run_of_them_together():
    """A model with the bias is trained on packed prompts, then serves: the prompts' scores without a cache, their keys stored, further
    tokens prefilled in a chunk and decoded one by one.  All agree with one pass over the whole sequences."""
    heads, hkv, d, block = 8, 2, 128, 16
    prompt, chunk, steps = np.array([70, 130]), 20, 3
    total = prompt + chunk + steps
    c = Case(total.tolist(), total.tolist(), heads, hkv, d, 0, 32, 128)
    out, lse, grads = both(c)
    check(c, out, lse, grads)
    c.bias -= 0.05 * grads[3]  # a step of training
    r = c.oracle(False)
    tol = paged_tolerance(c, r)
    p = Paged(c, block)
    p.k.zero_(), p.v.zero_()
    part = lambda t, a, b: torch.cat([t[int(s) + a[i]:int(s) + b[i]] for i, s in enumerate(c.cu_q[:-1])])  # noqa: E731
    pick = lambda x, a, b: np.concatenate([x[int(s) + a[i]:int(s) + b[i]] for i, s in enumerate(c.cu_q[:-1])])  # noqa: E731
    zero = [0, 0]
    got, _ = pa.pa_varlen_attn(part(c.q, zero, prompt), part(c.k, zero, prompt), part(c.v, zero, prompt), dev(offsets(prompt)),
                               dev(offsets(prompt)), 130, 130, c.scale, bias=c.bias, max_distance=128)
    within(got, pick(r["out"], zero, prompt), pick(tol, zero, prompt), "scores")
    pa.pa_store_kvcache(part(c.k, zero, prompt), part(c.v, zero, prompt), p.k, p.v, dev(pick(p.slots, zero, prompt)))
    have = prompt + chunk
    got = pa.pa_varlen_prefill_bias(part(c.q, prompt, have), p.k, p.v, dev([0, chunk, 2 * chunk]), dev(have), dev(p.table), chunk, 200,
                                    c.scale, c.bias, 128, key=part(c.k, prompt, have), value=part(c.v, prompt, have),
                                    slot_mapping=dev(pick(p.slots, prompt, have)))
    within(got, pick(r["out"], prompt, have), pick(tol, prompt, have), "chunk")
    for _ in range(steps):
        got = pa.pa_decode_bias(part(c.q, have, have + 1), p.k, p.v, dev(p.table), dev(have + 1), 200, c.scale, c.bias, 128,
                                key=part(c.k, have, have + 1), value=part(c.v, have, have + 1),
                                slot_mapping=dev(pick(p.slots, have, have + 1)))
        within(got, pick(r["out"], have, have + 1), pick(tol, have, have + 1), "decode")
        have = have + 1
    assert pa.pa_read_device_error() == 0
