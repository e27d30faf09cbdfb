"""Pins of the 4-bit cache's oracle and host-side refusals of its entry points (CPU)."""
import numpy as np
import pytest
import torch

import paged_kv_attention_03_gb300 as pa
from oracle import fp4

OK, INVALID, UNSUPPORTED = pa.PA_OK, pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED
FAKE, MISALIGNED = 0x10000, 0x10002  # never dereferenced on these paths


def test_e4m3_values_and_rounding_match_torch():
    codes = torch.arange(127, dtype=torch.uint8)
    np.testing.assert_array_equal(codes.view(torch.float8_e4m3fn).double().numpy(), fp4.E4M3)
    x = np.abs(np.random.default_rng(0).standard_normal(20000)).astype(np.float32) * 60
    x = np.minimum(x, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(fp4.nearest_code(x, fp4.E4M3), want)
    mid = (fp4.E4M3[1:] + fp4.E4M3[:-1]) / 2  # ties
    want = torch.from_numpy(mid).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(fp4.nearest_code(mid, fp4.E4M3), want)


def test_e2m1_rounding():
    # Halfway cases go to the even code; beyond 6 saturates.
    x = [0.0, 0.25, 0.26, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.1, 6.0, 100.0]
    assert list(fp4.nearest_code(np.array(x), fp4.E2M1)) == [0, 0, 1, 2, 2, 4, 4, 6, 6, 7, 7, 7]


@pytest.mark.parametrize("kv_scale", [1.0, 0.37])
def test_quantise_then_expand(kv_scale):
    x = torch.randn(50, 3, 64, generator=torch.Generator().manual_seed(1)).bfloat16().double().numpy()
    v = fp4.expand(fp4.quantise(x, kv_scale), kv_scale)
    top = np.abs(x.reshape(50, 3, 4, 16)).max(-1, keepdims=True)
    # The scale is within 2^-4 of max / 6 (E4M3 rounding); a code is off by at most half the
    # widest step of E2M1 (2 between 4 and 6), and the largest may saturate below 6 / (1 - 2^-4).
    bound = np.broadcast_to(top / 6 * (1 + 2.0 ** -4) * 1.0, (50, 3, 4, 16)).reshape(x.shape)
    assert (np.abs(v - x) <= bound * 1.0001).all()
    # Values that the format holds come back as they are.
    exact = np.array([0, .5, 1, 1.5, 2, 3, 4, 6] * 2, np.float64) * np.array([1, -1] * 8) * 0.25
    np.testing.assert_array_equal(fp4.expand(fp4.quantise(exact, 1.0), 1.0), exact)


def test_quantise_special_groups():
    z = np.zeros((1, 16))
    assert fp4.quantise(z, 1.0)[0, -1] == 1 and (fp4.expand(fp4.quantise(z, 1.0), 1.0) == 0).all()
    z[0, 3] = np.nan
    assert np.isnan(fp4.expand(fp4.quantise(z, 1.0), 1.0)).all()
    z[0, 3] = -np.inf
    v = fp4.expand(fp4.quantise(z, 1.0), 1.0)
    assert v[0, 3] == -6 * 448 and (np.delete(v, 3) == 0).all()


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.load()


def _store(lib, **kw):
    a = dict(key=FAKE, value=FAKE, kc=FAKE, vc=FAKE, slot=FAKE, n=3, nb=4, bs=16, hkv=2, d=64, s=1.0)
    a.update(kw)
    got = [fn(a["key"], a["value"], a["kc"], a["vc"], a["slot"], a["n"], a["nb"], a["bs"], a["hkv"],
              a["d"], a["s"], None) for fn in (lib.pa_store_kvcache_fp4, lib.pa_gather_kvcache_fp4)]
    assert got[0] == got[1]
    return got[0]


def test_store_and_gather_refusals(lib):
    assert _store(lib, n=0) == OK
    assert _store(lib, n=-1) == INVALID
    assert _store(lib, key=None) == INVALID
    assert _store(lib, vc=MISALIGNED) == INVALID
    for bs in (8, 24, 512):
        assert _store(lib, bs=bs) == UNSUPPORTED
    assert _store(lib, d=96) == UNSUPPORTED
    assert _store(lib, nb=1 << 28) == UNSUPPORTED
    for s in (0.0, -1.0, float("nan"), float("inf"), 1e-26, 1e26):
        assert _store(lib, s=s) == INVALID


def _decode(lib, **kw):
    a = dict(out=FAKE, q=FAKE, key=None, value=None, slot=None, kc=FAKE, vc=FAKE, bt=FAKE, mb=8,
             lens=FAKE, batch=2, most=100, nb=16, bs=16, H=8, Hkv=2, D=128, window=0, scale=0.1,
             kvs=1.0, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_decode_fp4(*a.values(), None)


def _prefill(lib, **kw):
    a = dict(out=FAKE, q=FAKE, key=None, value=None, slot=None, kc=FAKE, vc=FAKE, cuq=FAKE, cuk=None,
             lens=FAKE, bt=FAKE, mb=8, n=2, total=10, mq=8, mk=100, nb=16, bs=16, H=8, Hkv=2, D=128,
             window=0, scale=0.1, kvs=1.0, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_varlen_prefill_fp4(*a.values(), None)


@pytest.mark.parametrize("call", [_decode, _prefill])
def test_attention_refusals(lib, call):
    assert call(lib, H=9) == INVALID
    assert call(lib, H=130, Hkv=2) == UNSUPPORTED
    assert call(lib, D=96) == UNSUPPORTED
    assert call(lib, bs=8) == UNSUPPORTED
    assert call(lib, scale=0.0) == INVALID
    assert call(lib, scale=float("nan")) == INVALID
    assert call(lib, scale=float("inf")) == INVALID
    assert call(lib, scale=1e20, kvs=1e20) == INVALID
    assert call(lib, kvs=0.0) == INVALID
    assert call(lib, key=FAKE) == INVALID
    assert call(lib, q=None) == INVALID
    assert call(lib, kc=MISALIGNED) == INVALID
    assert call(lib, key=MISALIGNED, value=FAKE, slot=FAKE) == INVALID


def test_attention_empty_calls_and_workspace(lib):
    assert _decode(lib, batch=0) == OK and _decode(lib, batch=-1) == INVALID
    assert _decode(lib, batch=65536) == UNSUPPORTED
    assert _prefill(lib, total=0) == OK and _prefill(lib, n=0) == OK
    assert _prefill(lib, mq=200) == INVALID  # more queries than keys
    assert _decode(lib, most=2 ** 31 - 1) == UNSUPPORTED and _prefill(lib, mk=2 ** 31 - 1) == UNSUPPORTED
    assert _prefill(lib, lens=None) == INVALID
    # Short sequences need no workspace; long ones one of the advertised size and alignment.
    assert pa.pa_decode_fp4_workspace_size(4, 8, 2, 64, 100) == 0
    need = pa.pa_decode_fp4_workspace_size(2, 8, 2, 128, 4096)
    assert need > 0
    for call, most in ((_decode, "most"), (_prefill, "mk")):
        assert call(lib, **{most: 4096}) == INVALID
        assert call(lib, ws=FAKE, wsb=need - 1, **{most: 4096}) == INVALID
        assert call(lib, ws=FAKE + 16, wsb=need, **{most: 4096}) == INVALID
    assert pa.pa_decode_fp4_workspace_size(2, 6, 4, 128, 4096) == 0


def test_step_refusals(lib):
    def prepare(**kw):
        a = dict(bt=FAKE, lens=FAKE, cu=FAKE, slots=FAKE, pos=None, nfo=FAKE, ctx=FAKE, q=FAKE, free=FAKE,
                 nf=FAKE, n=2, mb=4, tokens=8, nb=16, bs=16)
        a.update(kw)
        return lib.pa_prepare_step(*a.values(), None)

    def release(**kw):
        a = dict(free=FAKE, nfo=FAKE, out=FAKE, fin=FAKE, lens=FAKE, bt=FAKE, nf=FAKE, n=2, mb=4, nb=16, bs=16)
        a.update(kw)
        return lib.pa_release_blocks(*a.values(), None)

    for call in (prepare, release):
        assert call(n=-1) == INVALID
        assert call(n=16385) == UNSUPPORTED
        assert call(bs=24) == UNSUPPORTED
        assert call(nb=1 << 28) == UNSUPPORTED
        assert call(bt=None) == INVALID
        assert call(nf=None) == INVALID
        assert call(mb=0) == INVALID
    assert prepare(tokens=-1) == INVALID
    assert prepare(cu=None) == INVALID
    assert prepare(slots=None) == INVALID
    assert release(fin=None) == INVALID


def test_binding_refuses_wrong_tensors():
    # CPU tensors, before anything is launched.
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_prepare_step(i, i, torch.zeros(2, 4, dtype=torch.int32), i, i[:1], 16, 8)
    c = torch.zeros(4, 2, 16, 72, dtype=torch.uint8)
    with pytest.raises(ValueError):
        pa.pa_gather_kvcache_fp4(c, c, i, 1.0)


@pytest.mark.parametrize("heads,hkv", [(8, 8), (32, 8), (40, 8), (14, 2), (64, 1)])
def test_prefill_workspace_for_a_query_length(lib, heads, hkv):
    # Up to two blocks of queries (of 2 floor(128 / group) tokens) a sequence: what the decode rows
    # need; longer ones: with the room for expanded keys.
    small = pa.pa_decode_fp4_workspace_size(4, heads, hkv, 128, 4096)
    full = pa.pa_varlen_prefill_fp4_workspace_size(4, heads, hkv, 128, 4096)
    assert 0 < small and full >= small + 2 * 2 * 4 * 4096 * hkv * 128
    edge = 4 * (128 // (heads // hkv))
    for most, want in ((0, small), (1, small), (edge, small), (edge + 1, full), (4096, full)):
        assert pa.pa_varlen_prefill_fp4_workspace_size(4, heads, hkv, 128, 4096, 0, most) == want
    assert pa.pa_varlen_prefill_fp4_workspace_size(4, heads, hkv, 128, 4096, 0, -1) == 0
    assert pa.pa_varlen_prefill_fp4_workspace_size(4, 9, 2, 128, 4096, 0, 4096) == 0


@pytest.mark.parametrize("new", [{}, dict(key=FAKE, value=FAKE, slot=FAKE)])
def test_prefill_refuses_sizes_before_it_stores(lib, new):
    # Sizes past the prefill's own counters are refused while nothing has been stored.
    need = 1 << 40
    big = dict(ws=FAKE, wsb=need, mb=1 << 20, **new)
    assert _prefill(lib, n=65535, mq=1 << 20, mk=1 << 20, H=64, Hkv=8, **big) == UNSUPPORTED  # 2^36 items
    assert _prefill(lib, nb=(1 << 27) - 16, bs=16, **big) == UNSUPPORTED  # 2^31 - 256 slots
    assert _prefill(lib, total=2 ** 31 - 256, **big) == UNSUPPORTED
