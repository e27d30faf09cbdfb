"""CPU checks of the relative-bias oracle (worked buckets, closed forms, differences) and of the refusals of the packed
and biased entry points, all of which happen on the host."""
import math
from fractions import Fraction

import numpy as np
import pytest

import paged_kv_attention_03_gb300 as pa
from oracle import relative

OK, INVALID, UNSUPPORTED = pa.PA_OK, pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
FAKE, MISALIGNED = 0x10000, 0x10002


def test_buckets_of_the_common_sizes():
    # 32 buckets up to 128: 16 exact ones, then borders at 16 * 8^(j / 16), rounded up
    first = relative.first_distances(32, 128)
    assert first[:17] == list(range(17))
    assert first[17:] == [math.ceil(16 * 8 ** (j / 16) - 1e-9) for j in range(1, 16)]
    # a border that is a whole number belongs to the bucket beyond it: 8 * 16^(2 / 8) = 16
    assert relative.first_distances(16, 128)[10] == 16
    assert relative.buckets(np.array([15, 16]), 16, 128).tolist() == [9, 10]


@pytest.mark.parametrize("num_buckets,max_distance", [(2, 2), (3, 7), (8, 9), (32, 17), (32, 128), (33, 500), (128, 32768)])
def test_the_table_knows_the_last_bucket(num_buckets, max_distance):
    """The library's table has bytes for last + 776 entries a head, a multiple of 4: its `last` is the oracle's."""
    last = relative.first_distances(num_buckets, max_distance)[-1]
    row = (last + 776 + 3) // 4 * 4
    assert pa.pa_relative_bias_workspace_size(64, num_buckets, max_distance) == 64 * row * 4
    m = num_buckets // 2
    r = num_buckets - m
    if r > 1:  # last - 1 lies before the border, last does not
        border = Fraction(max_distance, m) ** (r - 1)
        assert Fraction(last - 1, m) ** r < border <= Fraction(last, m) ** r


def test_gradient_against_differences():
    g = np.random.default_rng(0)
    cu_q, cu_k = [0, 5, 5, 9], [0, 7, 10, 12]  # more keys, no queries, more queries than keys
    q, k, v, w = (g.standard_normal(s) for s in ((9, 4, 3), (12, 2, 3), (12, 2, 3), (9, 4, 3)))
    bias = g.standard_normal((6, 4))
    for window in (0, 3):
        f = lambda q, k, v, bias: (relative.attention(q, k, v, cu_q, cu_k, window, 0.7, bias, 5)["out"] * w).sum()  # noqa: E731
        r = relative.attention(q, k, v, cu_q, cu_k, window, 0.7, bias, 5, dout=w)
        for at, name in enumerate(("dq", "dk", "dv", "dbias")):
            args = [q, k, v, bias]
            got = np.zeros(args[at].shape)
            for i in np.ndindex(got.shape):
                d = np.zeros(got.shape)
                d[i] = 1e-5
                up, down = list(args), list(args)
                up[at], down[at] = args[at] + d, args[at] - d
                got[i] = (f(*up) - f(*down)) / 2e-5
            # central differences: h^2 times third derivatives of order one, and 1e-16 / h of rounding
            np.testing.assert_allclose(np.nan_to_num(r[name]), got, atol=1e-8)
        assert (r["out"][5] == 0).all() and np.isneginf(r["lse"][5]).all()  # positions -2, -1
        assert abs(r["dbias"].sum(0)).max() < 1e-12  # a row's dS sum to zero


def _packed(lib, **kw):
    a = dict(out=FAKE, lse=FAKE, q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, cuq=FAKE, cuk=FAKE, n=2, tq=10, tk=12, mq=8,
             mk=9, H=8, Hkv=2, D=128, window=0, scale=0.1, bias=FAKE, nb=32, md=128, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.pa_varlen_attn(*a.values(), None)


def _backward(lib, **kw):
    a = dict(dq=FAKE, dk=FAKE, dv=FAKE, db=FAKE, dqs=1024, dks=256, dvs=256, dout=FAKE, q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=FAKE,
             qs=1024, ks=256, vs=256, cuq=FAKE, cuk=FAKE, n=2, tq=10, tk=12, mq=8, mk=9, H=8, Hkv=2, D=128, window=0, scale=0.1,
             bias=FAKE, nb=32, md=128, ws=None, ws_bytes=0)
    a.update(kw)
    return lib.pa_varlen_attn_backward(*a.values(), None)


@pytest.mark.parametrize("call", [_packed, _backward])
def test_packed_refusals(call):
    lib = pa.load()
    assert call(lib) == INVALID  # no workspace
    table = pa.pa_relative_bias_workspace_size(8, 32, 128)
    need = table if call is _packed else pa.pa_varlen_attn_backward_workspace_size(10, 12, 2, 8, 32, 128)
    assert need >= table > 0
    assert call(lib, ws=FAKE, ws_bytes=need - 1) == INVALID
    assert call(lib, ws=FAKE + 16, ws_bytes=need) == INVALID
    ws = dict(ws=FAKE, ws_bytes=1 << 40)
    for bad in (dict(q=None), dict(k=MISALIGNED), dict(v=None), dict(out=MISALIGNED), dict(cuq=None), dict(cuk=None), dict(lse=None),
                dict(H=6, Hkv=4), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(tq=-1), dict(mk=-1),
                dict(n=-1), dict(qs=1023), dict(qs=1016), dict(ks=260), dict(vs=0), dict(vs=-256), dict(nb=1), dict(nb=0), dict(md=16),
                dict(bias=None), dict(bias=MISALIGNED)):
        assert call(lib, **{**ws, **bad}) == INVALID, bad
    for bad in (dict(D=96, qs=768, ks=192, vs=192), dict(H=130, Hkv=2, qs=130 * 128), dict(nb=129, md=4000), dict(md=32769),
                dict(tq=1 << 30), dict(tk=1 << 30), dict(n=65536), dict(mq=1 << 30, n=60000)):
        assert call(lib, **{**ws, **bad}) == UNSUPPORTED, bad
    assert call(lib, n=0, bias=None, nb=0, **({} if call is _packed else {"db": None})) == OK
    if call is _backward:
        assert call(lib, **ws, db=None) == INVALID  # a bias and its gradient go together
        assert call(lib, **ws, bias=None, nb=0) == INVALID
        for bad in (dict(dq=None), dict(dk=None), dict(dv=MISALIGNED), dict(dout=None), dict(dqs=1000), dict(dks=128), dict(dvs=257)):
            assert call(lib, **{**ws, **bad}) == INVALID, bad


def test_paged_refusals():
    lib = pa.load()

    def decode(**kw):
        a = dict(out=FAKE, q=FAKE, key=None, value=None, slot=None, kc=FAKE, vc=FAKE, bt=FAKE, width=8, lens=FAKE, batch=2, most=100,
                 blocks=16, bs=16, H=8, Hkv=2, D=128, window=0, scale=0.1, bias=FAKE, nb=32, md=128, splits=1, ws=None, ws_bytes=0)
        a.update(kw)
        return lib.pa_decode_bias(*a.values(), None)

    def prefill(**kw):
        a = dict(out=FAKE, q=FAKE, key=None, value=None, slot=None, kc=FAKE, vc=FAKE, cuq=FAKE, cuk=None, lens=FAKE, bt=FAKE, width=8,
                 n=2, tq=10, mq=8, mk=100, blocks=16, bs=16, H=8, Hkv=2, D=128, window=0, scale=0.1, bias=FAKE, nb=32, md=128, ws=FAKE,
                 ws_bytes=1 << 30)
        a.update(kw)
        return lib.pa_varlen_prefill_bias(*a.values(), None)

    assert decode(batch=0) == OK and prefill(tq=0) == OK
    for call in (decode, prefill):
        for bad in (dict(bias=None), dict(nb=0), dict(md=16), dict(scale=0.0), dict(H=9), dict(q=None), dict(key=FAKE), dict(out=MISALIGNED),
                    dict(blocks=-1)):
            assert call(**bad) == INVALID, bad
        for bad in (dict(nb=200, md=1000), dict(md=40000), dict(scale=1e-21), dict(D=96), dict(H=130), dict(bs=24)):
            assert call(**bad) == UNSUPPORTED, bad
    assert decode(splits=4, most=4096) == INVALID  # needs a workspace
    assert prefill(ws=None) == INVALID and prefill(ws_bytes=100) == INVALID and prefill(ws=FAKE + 16) == INVALID
    assert prefill(bs=8) == UNSUPPORTED and prefill(mq=101) == INVALID and prefill(lens=None) == INVALID


def test_size_functions_of_unsupported_sizes():
    assert pa.pa_relative_bias_workspace_size(8, 1, 10) == 0
    assert pa.pa_relative_bias_workspace_size(8, 32, 16) == 0
    assert pa.pa_relative_bias_workspace_size(0, 32, 128) == 0
    assert pa.pa_varlen_attn_backward_workspace_size(-1, 10, 1, 8) == 0
    assert pa.pa_varlen_attn_backward_workspace_size(100, 90, 3, 8) > 0
