"""The 4-bit KV cache on the GPU against the fp64 oracle (oracle/fp4.py).

The store is bit-exact: its definition fixes every 32-bit operation and rounding.

Tolerance of the attention, element by element, with A = sum_j p_j |v_j| (the oracle's
`weight`), n keys and vmax the largest |v|:
  * the output's rounding to bf16: 2^-8 |ref| (half a step, finfo.eps / 2);
  * the softmax weights' rounding to f16: 2^-11 relative in the numerator and, through the
    denominator that sums the rounded weights, at most 2^-11 more: 2^-10 A; weights below
    2^-14 of the reference maximum are off by 2^-25 each at most, and the weights sum to
    2^-8 of ... at least 1 (the maximum's own weight is at least 1): n 2^-25 vmax each in
    numerator and denominator;
  * fp32 scores (products exact in fp32, sums of D terms: relative 2^-24 a term) move a weight
    by under 2^-13 for |scores| below 100 at D = 128: 2^-12 A with the denominator, which the
    fp32 sums of up to n rounded products (n 2^-24 A, n <= 4096 here) are inside of;
  * q is exact in f16 for |q| >= 2^-14 and off by 2^-25 below: under 2^-13 of a weight too.
"""
import numpy as np
import pytest
import torch

import paged_kv_attention_03_gb300 as pa
from oracle import fp4

pytestmark = pytest.mark.gpu

KVS = 0.7


def _t(a, dev):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)


def _bf(shape, seed, size=1.0):
    return (size * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).bfloat16()


class Case:
    """A packed step over a 4-bit cache whose every row holds a quantised N(0, 1)."""

    def __init__(self, dev, ctx, new, heads, kv_heads, dim, bs=16, seed=0, kv_scale=KVS):
        rng = np.random.default_rng(seed)
        self.dev, self.heads, self.dim, self.kv_scale = dev, heads, dim, kv_scale
        ctx, new = np.asarray(ctx), np.asarray(new)
        self.lens, self.new = ctx + new, new
        blocks = -(-self.lens // bs)
        nb = int(blocks.sum()) + 3
        perm = rng.permutation(nb)
        self.table = np.full((len(ctx), max(int(blocks.max()), 1) + 1), -1, np.int32)
        at = 0
        for i, n in enumerate(blocks):
            self.table[i, :n] = perm[at:at + n]
            at += int(n)
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        tq = int(self.cu[-1])
        self.slots = np.concatenate([[self.table[i, p // bs] * bs + p % bs for p in range(c, c + n)]
                                     for i, (c, n) in enumerate(zip(ctx, new))] + [[]]).astype(np.int32)
        self.q = _bf((tq, heads, dim), seed + 1)
        self.key, self.value = _bf((tq, kv_heads, dim), seed + 2), _bf((tq, kv_heads, dim), seed + 3)
        quant = lambda k: fp4.quantise(_bf((nb, kv_heads, bs, dim), seed + k).double().numpy(), kv_scale)  # noqa: E731
        self.kc, self.vc = quant(4), quant(5)
        self.scale = dim ** -0.5
        self.bs = bs

    def device(self):
        d = self.dev
        return dict(q=self.q.to(d), k_cache=torch.from_numpy(self.kc).to(d), v_cache=torch.from_numpy(self.vc).to(d),
                    block_table=_t(self.table, d), seq_lens=_t(self.lens, d))

    def new_tokens(self):
        return dict(key=self.key.to(self.dev), value=self.value.to(self.dev), slot_mapping=_t(self.slots, self.dev))

    def store(self):
        """The oracle's store of the step's new tokens."""
        fp4.store(self.key.double().numpy(), self.kc, self.slots, self.kv_scale)
        fp4.store(self.value.double().numpy(), self.vc, self.slots, self.kv_scale)

    def decode(self, window=0, **kw):
        kw = dict(kw) if "q" in kw else {**self.device(), **kw}
        return pa.pa_decode_fp4(kw.pop("q"), kw.pop("k_cache"), kw.pop("v_cache"), kw.pop("block_table"),
                                kw.pop("seq_lens"), max(self.lens.max(), np.int64(0)), self.scale, self.kv_scale, window, **kw)

    def prefill(self, window=0, lens=True, cu_k=False, expand=True, **kw):
        """expand False: a workspace without room for the expanded keys, so that every query block
        expands its tiles itself; True: the declared maximum of the query lengths is so large that
        the keys are expanded beforehand whatever the lengths."""
        x = dict(kw) if "q" in kw else {**self.device(), **kw}
        sl = x.pop("seq_lens")
        most = max(128 * 6 if expand else 0, int(self.new.max()))
        if not expand:
            need = pa.pa_decode_fp4_workspace_size(len(self.lens), self.heads, self.kc.shape[1], self.dim, int(self.lens.max()),
                                                   window)
            x["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device=self.dev)
        if cu_k:
            x["cu_seqlens_k"] = _t(np.concatenate([[0], np.cumsum(self.lens)]), self.dev)
        return pa.pa_varlen_prefill_fp4(x.pop("q"), x.pop("k_cache"), x.pop("v_cache"), _t(self.cu, self.dev),
                                        sl if lens else None, x.pop("block_table"), most,
                                        max(most, int(self.lens.max())), self.scale, self.kv_scale, window, **x)

    def check(self, out, window=0, rows=None):
        assert pa.pa_read_device_error(device=self.dev) == 0
        ref, weight = fp4.paged_attention(self.q.double().numpy(), self.kc, self.vc, self.cu, self.lens, self.table,
                                          self.heads, window, self.scale, self.kv_scale)
        got = out.double().cpu().numpy()
        assert np.isfinite(got).all()
        vmax = 6 * 448 * self.kv_scale if not weight.size else np.abs(fp4.expand(self.vc, self.kv_scale)).max()
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2.0 ** -12) * weight + 2 * int(self.lens.max()) * 2.0 ** -25 * vmax
        err = np.abs(got - ref)
        worst = float((err / tol).max()) if err.size else 0.0
        assert worst <= 1, f"error {float(err.max()):.3e}, {worst:.2f} of the tolerance"


# ------------------------------------------------------------------- store ---
@pytest.mark.parametrize("dim,hkv,bs", [(128, 8, 16), (64, 2, 64), (128, 1, 256), (64, 3, 32)])
@pytest.mark.parametrize("tokens", [1, 5, 333])
def test_store_is_bit_exact_and_gather_reads_it_back(cuda, dim, hkv, bs, tokens):
    rng = np.random.default_rng(tokens)
    nb = -(-tokens // bs) + 3
    g = torch.Generator().manual_seed(dim)
    # Magnitudes from far below the smallest scale to saturation.
    size = torch.tensor([1e-30, 1e-4, 1e-2, 1.0, 30.0, 5000.0])[torch.randint(0, 6, (tokens, hkv, dim // 16), generator=g)]
    x = [(torch.randn(tokens, hkv, dim, generator=g) * size.repeat_interleave(16, -1)).bfloat16() for _ in range(2)]
    x[0][0, 0, :16] = 0
    slots = rng.permutation(nb * bs)[:tokens].astype(np.int32)
    slots[rng.random(tokens) < 0.2] = -1
    host = [rng.integers(0, 256, (nb, hkv, bs, dim // 2 + dim // 16)).astype(np.uint8) for _ in range(2)]
    dev = [torch.from_numpy(h).to(cuda) for h in host]
    pa.pa_store_kvcache_fp4(x[0].to(cuda), x[1].to(cuda), *dev, _t(slots, cuda), KVS)
    key, value = pa.pa_gather_kvcache_fp4(*dev, _t(slots, cuda), KVS)
    assert pa.pa_read_device_error(device=cuda) == 0
    for h, d, v, back in zip(host, dev, x, (key, value)):
        fp4.store(v.double().numpy(), h, slots, KVS)
        np.testing.assert_array_equal(d.cpu().numpy(), h)
        rows = np.zeros(v.shape)
        ok = slots >= 0
        rows[ok] = fp4.expand(h[slots[ok] // bs, :, slots[ok] % bs], KVS)
        # code * scale is exact; times kv_scale is one fp32 rounding, then one to bf16
        want = torch.from_numpy(rows.astype(np.float32)).bfloat16()
        assert torch.equal(back.cpu(), want)
    # Outputs that are aligned to 16 bytes only.
    n = key.numel()
    buf = torch.zeros(2, n + 16, dtype=torch.bfloat16, device=cuda)
    odd = [b[8:8 + n].view(key.shape) for b in buf]
    pa.pa_gather_kvcache_fp4(*dev, _t(slots, cuda), KVS, key=odd[0], value=odd[1])
    assert torch.equal(odd[0], key) and torch.equal(odd[1], value) and (buf[:, :8] == 0).all() and (buf[:, 8 + n:] == 0).all()


def test_store_ties_and_special_values(cuda):
    # kv_scale 1 and a largest element of 6 give scale 1: every halfway case of E2M1, both signs;
    # a NaN makes its group NaN, an infinity saturates, other groups stay.
    x = torch.zeros(3, 1, 64)
    x[0, 0, :16] = torch.tensor([6, .25, .75, 1.25, 1.75, 2.5, 3.5, 5, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5, -6])
    x[1, 0, 5], x[1, 0, 20] = float("nan"), 1.0
    x[2, 0, 5], x[2, 0, 6], x[2, 0, 40] = float("-inf"), 2.0, 1.0
    x = x.bfloat16()
    k = torch.zeros(1, 1, 16, 36, dtype=torch.uint8, device=cuda)
    v = torch.zeros_like(k)
    slots = _t([2, 0, 9], cuda)
    pa.pa_store_kvcache_fp4(x.to(cuda), x.to(cuda), k, v, slots, 1.0)
    got, _ = pa.pa_gather_kvcache_fp4(k, v, slots, 1.0)
    assert pa.pa_read_device_error(device=cuda) == 0
    want = fp4.expand(fp4.quantise(x.double().numpy(), 1.0), 1.0)
    np.testing.assert_array_equal(got.double().cpu().numpy(), want)
    assert want[0, 0, 1:8].tolist() == [0, 1, 1, 2, 2, 4, 4] and np.isnan(want[1, 0, :16]).all()
    # 1 alone: scale E4M3(1 / 6) = 11 / 64, code E2M1(64 / 11 = 5.82) = 6, and 6 * 11 / 64 = 1.03125
    assert want[2, 0, 5] == -6 * 448 and want[2, 0, 40] == 1.03125


@pytest.mark.parametrize("kv_scale", [1.0, 1 / 3, 1e-25, 3.7e-24, 1e25, 7.3e24, 0.0117, 271.828])
def test_store_rounds_every_quotient(cuda, kv_scale):
    # Every bf16 significand at every distance from its group's largest value, for scales with few
    # and with all bits: codes and scales equal the oracle's, whose divisions are fp32 ones.
    g = torch.Generator().manual_seed(1)
    kvs = float(np.float32(kv_scale))
    x = torch.randint(128, 256, (4000, 2, 64), generator=g).double() * 2.0 ** torch.randint(-12, 1, (4000, 2, 64), generator=g).double()
    x = (x * torch.where(torch.rand(x.shape, generator=g) < 0.5, -1.0, 1.0) * kvs *
         2.0 ** torch.randint(-12, 7, (4000, 2, 1), generator=g).double()).float().bfloat16()
    host = np.zeros((250, 2, 16, 36), np.uint8)
    k = torch.from_numpy(host.copy()).to(cuda)
    v = torch.zeros_like(k)
    pa.pa_store_kvcache_fp4(x.to(cuda), x.to(cuda), k, v, torch.arange(4000, dtype=torch.int32, device=cuda), kv_scale)
    fp4.store(x.double().numpy(), host, np.arange(4000), kv_scale)
    np.testing.assert_array_equal(k.cpu().numpy(), host)
    assert torch.equal(k, v)


def test_store_and_gather_flag_slots_past_the_pool(cuda):
    x = _bf((3, 2, 64), 1).to(cuda)
    buf = torch.zeros(3, 2, 16, 36, dtype=torch.uint8, device=cuda)  # a block behind the caches
    k, v = buf[:1], buf[1:2]
    pa.pa_store_kvcache_fp4(x, x, k, v, _t([16, 1000000, 3], cuda), 1.0)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_SLOT_RANGE
    assert (buf[2] == 0).all() and (k[0, :, :3] == 0).all() and (k[0, :, 4:] == 0).all()
    key, _ = pa.pa_gather_kvcache_fp4(k, v, _t([16, -1, 3], cuda), 1.0)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_SLOT_RANGE
    assert (key[:2] == 0).all() and (key[2] != 0).any()


# ------------------------------------------------------------------ decode ---
HEADS = [(32, 8), (40, 8), (8, 8), (14, 2), (16, 2), (18, 2), (16, 1), (64, 1)]


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("heads,kv_heads", HEADS)
def test_decode_head_layouts(cuda, heads, kv_heads, dim):
    c = Case(cuda, [0, 15, 16, 200, 777], [1] * 5, heads, kv_heads, dim, seed=heads)
    c.check(c.decode())


@pytest.mark.parametrize("window", [0, 1, 15, 16, 17, 100, 5000])
@pytest.mark.parametrize("bs", [16, 32, 128, 256])
def test_decode_lengths_and_windows(cuda, window, bs):
    c = Case(cuda, [0, 1, 14, 15, 16, 17, 127, 128, 129, 300, 1000, 2049], [1] * 12, 8, 2, 128, bs=bs, seed=bs)
    c.check(c.decode(window), window)


@pytest.mark.parametrize("lens", [[1], [16], [17], [100, 3], [144], [33, 64, 17, 100], [1] * 70, [90] * 700])
def test_decode_short_sequences(cuda, lens):
    # Up to 144 keys: whole segments, one launch, no workspace.
    c = Case(cuda, np.array(lens) - 1, [1] * len(lens), 8, 2, 64, seed=len(lens))
    assert pa.pa_decode_fp4_workspace_size(len(lens), 8, 2, 64, int(c.lens.max())) == 0
    c.check(c.decode())


@pytest.mark.parametrize("batch", [1, 2, 127, 128, 129, 300])
def test_decode_batches(cuda, batch):
    # Ragged lengths, sequences without keys among them (zero rows).
    rng = np.random.default_rng(batch)
    c = Case(cuda, rng.integers(-1, 400, batch), [1] * batch, 10, 2, 128, seed=batch)
    c.lens[0] = 399
    c = Case(cuda, c.lens - 1, [1] * batch, 10, 2, 128, seed=batch)
    out = c.decode()
    c.check(out)
    assert (out[torch.from_numpy(c.lens == 0).to(cuda)] == 0).all()


def test_decode_long(cuda):
    c = Case(cuda, [4095, 3000], [1, 1], 5, 1, 128, seed=9)
    c.check(c.decode())


@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_decode_flat_and_peaked_softmax(cuda, size):
    c = Case(cuda, [500, 31], [1, 1], 8, 2, 128, seed=11)
    c.q = (c.q.float() * size).bfloat16()
    if size > 1:  # scores beyond the derivation's |score| < 100: keep them inside it
        c.scale /= 4
    c.check(c.decode())


@pytest.mark.parametrize("window", [0, 20])
def test_decode_ignores_rows_outside_the_range(cuda, window):
    # NaN scales and any codes behind the last key, before the window and in unused blocks.
    c = Case(cuda, [36, 4, 600], [1, 1, 1], 8, 2, 128, seed=12)
    dirty = [torch.from_numpy(c.kc.copy()).to(cuda), torch.from_numpy(c.vc.copy()).to(cuda)]
    seen = np.zeros(c.kc.shape[:1] + c.kc.shape[2:3], bool)
    for i, n in enumerate(c.lens):
        for p in range(max(0, n - window) if window else 0, n):
            seen[c.table[i, p // 16], p % 16] = True
    hide = torch.from_numpy(~seen).to(cuda)[:, None, :, None].expand(dirty[0].shape)
    for d in dirty:
        d[hide] = 0xff
    c.check(c.decode(window, k_cache=dirty[0], v_cache=dirty[1]), window)


@pytest.mark.parametrize("dim,heads,kv_heads", [(128, 32, 8), (64, 8, 2), (128, 36, 1)])
@pytest.mark.parametrize("ctx", [[0, 15, 16, 99], [40, 700, 1, 2047]])
def test_decode_stores_the_new_tokens(cuda, dim, heads, kv_heads, ctx):
    c = Case(cuda, ctx, [1] * 4, heads, kv_heads, dim, seed=13)
    c.slots[1] = -1  # one request brings none: its last key is what the cache holds
    x = c.device()
    out = c.decode(**x, **c.new_tokens())
    c.store()
    np.testing.assert_array_equal(x["k_cache"].cpu().numpy(), c.kc)
    np.testing.assert_array_equal(x["v_cache"].cpu().numpy(), c.vc)
    c.check(out)


def test_decode_flags_bad_slots(cuda):
    # A slot that is not the last key's (written, flagged), one past the pool (skipped), and a
    # new token of a sequence without keys (written, flagged).
    c = Case(cuda, [40, 50, 60], [1, 1, 1], 8, 2, 128, seed=14)
    for slot, flag in (((c.table[0, 0] * 16 + 3), pa.DEVERR_SLOT_MISMATCH), (c.kc.shape[0] * 16, pa.DEVERR_SLOT_RANGE)):
        x, new = c.device(), c.new_tokens()
        new["slot_mapping"][0] = int(slot)
        c.decode(**x, **new)
        assert pa.pa_read_device_error(device=cuda) == flag
        kc = c.kc.copy()
        fp4.store(c.key.double().numpy(), kc, new["slot_mapping"].cpu().numpy(), KVS)
        np.testing.assert_array_equal(x["k_cache"].cpu().numpy(), kc)
    x, new = c.device(), c.new_tokens()
    x["seq_lens"][2] = 0
    out = c.decode(**x, **new)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_SLOT_MISMATCH
    kc = c.kc.copy()
    fp4.store(c.key.double().numpy(), kc, c.slots, KVS)
    np.testing.assert_array_equal(x["k_cache"].cpu().numpy(), kc)
    assert (out[2] == 0).all()


def test_decode_flags_lengths_and_blocks(cuda):
    c = Case(cuda, [40, 500, 60], [1, 1, 1], 8, 2, 128, seed=15)
    x = c.device()
    x["seq_lens"][1] = 10 ** 6  # truncated to the declared maximum (501)
    x["seq_lens"][0] = -4
    out = c.decode(**x)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_SEQ_RANGE
    assert (out[0] == 0).all()
    # (Where a sequence is cut depends on the others' lengths, so its last bits may too.)
    lens, c.lens = c.lens, np.array([0, 501, 61])
    c.check(out)
    c.lens = lens
    x = c.device()
    x["block_table"][1, 2], x["block_table"][1, 7] = -1, c.kc.shape[0]
    out = c.decode(**x)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE
    # The bad blocks read as zeros.
    kc, vc = c.kc, c.vc
    zero = np.zeros((1,) + kc.shape[1:], np.uint8)
    c.kc, c.vc = np.concatenate([kc, zero]), np.concatenate([vc, zero])
    c.table[1, 2] = c.table[1, 7] = kc.shape[0]
    c.check(out)


def test_decode_nan_reaches_its_rows_only(cuda):
    c = Case(cuda, [200, 300], [1, 1], 8, 2, 128, seed=16)
    x = c.device()
    x["v_cache"][int(c.table[1, 3]), 1, 5, 64] = 0x7f  # scale of dims 0 .. 15, kv head 1
    out = c.decode(**x)
    good = c.decode()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[1, 4:, :16] = True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], good[~bad])


def test_decode_is_deterministic_and_leaves_other_rows(cuda):
    c = Case(cuda, [300, 4000, 50, 9], [1] * 4, 40, 8, 128, seed=17)
    first = c.decode()
    for _ in range(3):
        assert torch.equal(c.decode(), first)
    buf = torch.full((6, 40, 128), 7.0, dtype=torch.bfloat16, device=cuda)
    c.decode(out=buf[1:5])
    assert torch.equal(buf[1:5], first) and (buf[0] == 7).all() and (buf[5] == 7).all()


def test_calls_refuse_wrong_tensors(cuda):
    c = Case(cuda, [300, 40], [1, 1], 8, 2, 128, seed=19)
    x = c.device()
    for name, bad, error in (("q", x["q"].half(), TypeError), ("k_cache", x["k_cache"][..., :36], ValueError),
                             ("v_cache", x["v_cache"][:2], ValueError), ("seq_lens", x["seq_lens"][:1], ValueError),
                             ("block_table", x["block_table"].cpu(), ValueError)):
        with pytest.raises(error):
            c.decode(**{**x, name: bad})
        with pytest.raises(error):
            c.prefill(**{**x, name: bad})
    with pytest.raises(ValueError, match="together"):
        c.decode(**x, key=c.key.to(cuda))
    with pytest.raises(pa.PAError) as e:  # a workspace that is too small
        c.decode(**x, workspace=torch.empty(256, dtype=torch.uint8, device=cuda))
    assert e.value.status == pa.PA_ERR_INVALID_ARG


def test_decode_ignores_what_its_workspace_holds(cuda):
    c = Case(cuda, [300, 4000, 50, 9], [1] * 4, 32, 8, 128, seed=18)
    good = c.decode()
    need = pa.pa_decode_fp4_workspace_size(4, 32, 8, 128, 4001)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=cuda)
    assert torch.equal(c.decode(workspace=ws[:need]), good) and (ws[need:] == 0xff).all()


# ----------------------------------------------------------------- prefill ---
both = pytest.mark.parametrize("expand", [True, False])


@both
@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("heads,kv_heads", HEADS)
def test_prefill_head_layouts(cuda, heads, kv_heads, dim, expand):
    c = Case(cuda, [0, 15, 100], [40, 430, 2], heads, kv_heads, dim, seed=heads)
    c.check(c.prefill(expand=expand))


@both
@pytest.mark.parametrize("window", [0, 1, 60, 128, 400])
@pytest.mark.parametrize("bs", [16, 64, 256])
def test_prefill_chunks_and_windows(cuda, window, bs, expand):
    c = Case(cuda, [0, 0, 37, 130, 500, 3], [1, 160, 64, 129, 31, 1], 8, 2, 128, bs=bs, seed=20)
    c.check(c.prefill(window, expand=expand), window)


@both
@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("n", [2, 16, 63, 64, 65, 127, 128, 129, 255, 257, 700])
def test_prefill_tile_edges(cuda, n, dim, expand):
    c = Case(cuda, [0, 5], [n, n // 2 + 1], 8, 2, dim, seed=n)
    c.check(c.prefill(expand=expand))


@both
@pytest.mark.parametrize("n", [33, 200])
def test_prefill_without_seq_lens(cuda, n, expand):
    c = Case(cuda, [0, 20, 9], [n, 1, 60], 8, 2, 128, seed=21)
    c.check(c.prefill(lens=False, cu_k=True, expand=expand))
    c.check(c.prefill(cu_k=True, expand=expand))


@both
@pytest.mark.parametrize("new", [[1] * 5, [300, 1, 1, 200, 1], [0, 1, 0, 17, 0]])
@pytest.mark.parametrize("dim", [128, 64])
def test_prefill_mixed_batches_store_their_tokens(cuda, new, dim, expand):
    c = Case(cuda, [1000, 0, 37, 90, 600], new, 32, 8, dim, seed=22)
    x = c.device()
    out = c.prefill(expand=expand, **x, **c.new_tokens())
    c.store()
    np.testing.assert_array_equal(x["k_cache"].cpu().numpy(), c.kc)
    np.testing.assert_array_equal(x["v_cache"].cpu().numpy(), c.vc)
    c.check(out)


@both
@pytest.mark.parametrize("dim", [128, 64])
def test_prefill_ignores_rows_behind_the_last_key(cuda, dim, expand):
    c = Case(cuda, [0, 7], [37, 235], 8, 2, dim, seed=23)
    dirty = [torch.from_numpy(x.copy()).to(cuda) for x in (c.kc, c.vc)]
    for d in dirty:
        for i, n in enumerate(c.lens):
            if n % 16:
                d[int(c.table[i, n // 16]), :, int(n % 16):] = 0xff  # NaN scales
    c.check(c.prefill(k_cache=dirty[0], v_cache=dirty[1], expand=expand))


def test_prefill_ignores_what_its_workspace_holds(cuda):
    # The scratch cache starts as NaN: keys before a window's first tile and behind the last key
    # stay that.
    c = Case(cuda, [700, 7, 30], [300, 130, 1], 8, 2, 128, seed=26)
    for window in (0, 100):
        need = pa.pa_varlen_prefill_fp4_workspace_size(3, 8, 2, 128, 1000, window)
        ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=cuda)
        c.check(c.prefill(window, workspace=ws[:need]), window)
        assert (ws[need:] == 0xff).all()


@both
def test_prefill_flags_bad_blocks(cuda, expand):
    c = Case(cuda, [0, 7], [300, 130], 8, 2, 128, seed=24)
    x = c.device()
    x["block_table"][0, 2] = -1
    x["block_table"][1] = c.kc.shape[0]
    out = c.prefill(expand=expand, **x)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE
    zero = np.zeros((1,) + c.kc.shape[1:], np.uint8)
    c.kc, c.vc = np.concatenate([c.kc, zero]), np.concatenate([c.vc, zero])
    c.table[0, 2] = c.kc.shape[0] - 1
    c.table[1] = c.kc.shape[0] - 1
    c.check(out)


def test_prefill_wait_limit_runs_out_then_device_is_usable(cuda):
    c = Case(cuda, [0, 30], [200, 64], 8, 2, 128, seed=25)
    pa.pa_debug_prefill_stall(True, 20_000_000)
    try:
        c.prefill()
        flags = pa.pa_read_device_error(clear=True, device=cuda)
    finally:
        pa.pa_debug_prefill_stall(False, 0)
    assert flags & pa.DEVERR_TIMEOUT
    c.check(c.prefill())


def test_caches_beyond_four_gigabytes(cuda):
    # Every block of the step lies past byte 2^32 of both caches.
    c = Case(cuda, [300, 20, 0], [1, 200, 1], 8, 8, 128, seed=27)
    nb, row = c.kc.shape[0], 8 * 16 * 72
    first = (2 ** 32 + row) // row + 1
    big = [torch.empty(first + nb, 8, 16, 72, dtype=torch.uint8, device=cuda) for _ in range(2)]
    for b, h in zip(big, (c.kc, c.vc)):
        b[first:] = torch.from_numpy(h).to(cuda)
    x = c.device()
    x |= {"k_cache": big[0], "v_cache": big[1], "block_table": torch.where(x["block_table"] >= 0, x["block_table"] + first, -1)}
    new = c.new_tokens()
    new["slot_mapping"] = new["slot_mapping"] + first * 16
    for expand in (True, False):
        out = c.prefill(expand=expand, **x, **new)
    c.store()
    for b, h in zip(big, (c.kc, c.vc)):
        np.testing.assert_array_equal(b[first:].cpu().numpy(), h)
    c.check(out)
    key, value = pa.pa_gather_kvcache_fp4(*big, new["slot_mapping"], KVS)
    want = pa.pa_gather_kvcache_fp4(big[0][first:], big[1][first:], _t(c.slots, cuda), KVS)
    assert torch.equal(key, want[0]) and torch.equal(value, want[1])
    # The decode of the first and last sequence.
    rows = [0, 2]
    d = Case.__new__(Case)
    d.__dict__ = dict(c.__dict__)
    d.q, d.key, d.value = (t[[int(c.cu[i]) for i in rows]] for t in (c.q, c.key, c.value))
    d.lens, d.new, d.table, d.cu = c.lens[rows], c.new[rows], c.table[rows], np.array([0, 1, 2], np.int32)
    y = d.device() | {"k_cache": big[0], "v_cache": big[1]}
    y["block_table"] = torch.where(y["block_table"] >= 0, y["block_table"] + first, -1)
    d.check(d.decode(**y))


# ------------------------------------------------------ streams and graphs ---
def test_calls_on_two_streams_at_once(cuda):
    a = Case(cuda, [300, 4000, 50], [1] * 3, 32, 8, 128, seed=30)
    b = Case(cuda, [0, 500, 9], [200, 1, 77], 32, 8, 128, seed=31)
    xa, xb = a.device(), b.device()
    ga, gb = a.decode(**xa), b.prefill(**xb)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            torch.cuda._sleep(100000)
            got.append((ga, a.decode(**xa)))
        with torch.cuda.stream(s2):
            torch.cuda._sleep(100000)
            got.append((gb, b.prefill(**xb)))
    torch.cuda.synchronize()
    assert all(torch.equal(w, g) for w, g in got)


def test_decode_in_a_graph_follows_its_lengths(cuda):
    c = Case(cuda, [300, 1000, 50, 0], [1] * 4, 32, 8, 128, seed=32)
    x = c.device()
    out = torch.empty_like(x["q"])
    ws = torch.empty(pa.pa_decode_fp4_workspace_size(4, 32, 8, 128, 1001), dtype=torch.uint8, device=cuda)
    c.decode(**x, out=out, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.decode(**x, out=out, workspace=ws)
    for lens in ([301, 1001, 51, 1], [17, 1001, 0, 1], [1, 1, 1, 1], [300, 2, 30, 0]):
        x["seq_lens"].copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(float("nan"))
        graph.replay()
        c.lens = np.array(lens)
        c.new = np.ones(4, np.int64)
        c.check(out)


@pytest.mark.parametrize("captured", [False, True])
def test_decode_waits_for_what_precedes_it(cuda, captured):
    # Its inputs come from a copy, a kernel and another stream's kernels right before it; two calls
    # in a row share a workspace.
    c = Case(cuda, [300, 1000, 50, 9], [1] * 4, 32, 8, 128, seed=33)
    d = Case(cuda, [900, 10, 500, 70], [1] * 4, 32, 8, 128, seed=34)
    x, y = c.device(), d.device()
    want = [c.decode(**x), d.decode(**y)]
    ws = torch.empty(pa.pa_decode_fp4_workspace_size(4, 32, 8, 128, 1001), dtype=torch.uint8, device=cuda)
    q, lens, table = torch.empty_like(x["q"]), torch.empty_like(x["seq_lens"]), torch.empty_like(x["block_table"])
    out = [torch.empty_like(q), torch.empty_like(q)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())

    def step():
        if not captured:
            torch.cuda._sleep(2_000_000)
        q.zero_()
        lens.copy_(x["seq_lens"])
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mul(x["q"], 1, out=q)
            table.copy_(x["block_table"])
        torch.cuda.current_stream().wait_stream(side)
        c.decode(**{**x, "q": q, "seq_lens": lens, "block_table": table}, out=out[0], workspace=ws)
        d.decode(**y, out=out[1], workspace=ws)
        lens.zero_()
        table.fill_(-1)
        q.fill_(float("nan"))

    with torch.cuda.stream(main):
        step()
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                step()
    for _ in range(5):
        with torch.cuda.stream(main):
            for o in out:
                o.fill_(0)
            graph.replay() if captured else step()
            got = [o.clone() for o in out]
        torch.cuda.synchronize()
        assert pa.pa_read_device_error(device=cuda) == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@both
@pytest.mark.parametrize("captured", [False, True])
def test_prefill_waits_for_what_precedes_it(cuda, captured, expand):
    # The cache and the tables arrive by copies right before the call and are wiped right after it;
    # calls in a row share the workspace and its scratch cache.
    c = Case(cuda, [300, 0, 50, 9], [200, 300, 1, 33], 8, 2, 128, seed=35)
    x = c.device()
    most = 768 if expand else 300
    cu = _t(c.cu, cuda)
    need = pa.pa_varlen_prefill_fp4_workspace_size(4, 8, 2, 128, 768) if expand else \
        pa.pa_decode_fp4_workspace_size(4, 8, 2, 128, 768)
    ws = torch.empty(need, dtype=torch.uint8, device=cuda)
    y = {k: torch.empty_like(v) for k, v in x.items()}
    out = torch.empty_like(x["q"])

    def step():
        if not captured:
            torch.cuda._sleep(1_000_000)
        for k in x:
            y[k].copy_(x[k])
        for _ in range(2):
            pa.pa_varlen_prefill_fp4(y["q"], y["k_cache"], y["v_cache"], cu, y["seq_lens"], y["block_table"], most, 768,
                                     c.scale, c.kv_scale, out=out, workspace=ws)
        for k in ("k_cache", "v_cache", "q"):
            y[k].zero_()
        y["block_table"].fill_(-1)

    main = torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(main):
        step()
        torch.cuda.synchronize()
        c.check(out)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                step()
        for _ in range(3):
            out.fill_(float("nan"))
            graph.replay() if captured else step()
        torch.cuda.synchronize()
    c.check(out)


def test_a_serving_loop(cuda):
    """Lengths -> tables and slots -> prefill with its store -> decode steps -> release, one run
    of them together; every step's outputs against the oracle on the oracle's own cache."""
    bs, hkv, heads, dim, n, mb = 16, 2, 8, 128, 6, 20
    nb = 70
    rng = np.random.default_rng(40)
    free = rng.permutation(nb).astype(np.int32)
    table, lens, nf = np.full((n, mb), -1, np.int32), np.zeros(n, np.int64), nb
    kc = np.zeros((nb, hkv, bs, 72), np.uint8)
    vc = kc.copy()
    d_table, d_free, d_nf, d_lens = _t(table, cuda), _t(free, cuda), _t([nf], cuda), _t(lens, cuda)
    d_kc, d_vc = torch.zeros(kc.shape, dtype=torch.uint8, device=cuda), torch.zeros(vc.shape, dtype=torch.uint8, device=cuda)
    for step, new in enumerate(([70, 1, 33, 100, 0, 16], [1, 40, 1, 1, 9, 1], [1] * 6, None, [1, 60, 1, 1, 1, 50], [1] * 6)):
        if new is None:
            fin = np.array([0, 1, 0, 0, 0, 1], np.int32)
            pa.pa_release_blocks(_t(fin, cuda), d_lens, d_table, d_free, d_nf, bs, seq_lens_out=d_lens, num_free_out=d_nf)
            free, lens, nf = fp4.release_blocks(fin, lens, table, d_free.cpu().numpy(), nf, bs)
            continue
        tq = sum(new)
        _, cu, slots, _, _ = pa.pa_prepare_step(d_lens, _t(new, cuda), d_table, d_free, d_nf, bs, tq, seq_lens=d_lens,
                                                num_free_out=d_nf)
        table, lens, w_cu, w_slots, _, nf = fp4.prepare_step(lens, new, table, free, nf, bs, tq)
        q, k, v = _bf((tq, heads, dim), 50 + step), _bf((tq, hkv, dim), 60 + step), _bf((tq, hkv, dim), 70 + step)
        kw = dict(key=k.to(cuda), value=v.to(cuda), slot_mapping=slots)
        if max(new) > 1:
            out = pa.pa_varlen_prefill_fp4(q.to(cuda), d_kc, d_vc, cu, d_lens, d_table, max(new), mb * bs, dim ** -0.5, KVS, **kw)
        else:
            out = pa.pa_decode_fp4(q.to(cuda), d_kc, d_vc, d_table, d_lens, mb * bs, dim ** -0.5, KVS, **kw)
        fp4.store(k.double().numpy(), kc, w_slots, KVS)
        fp4.store(v.double().numpy(), vc, w_slots, KVS)
        assert pa.pa_read_device_error(device=cuda) == 0
        np.testing.assert_array_equal(d_kc.cpu().numpy(), kc)
        ref, weight = fp4.paged_attention(q.double().numpy(), kc, vc, w_cu, lens, table, heads, 0, dim ** -0.5, KVS)
        tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + 2.0 ** -12) * weight + 2 * mb * bs * 2.0 ** -25 * 10
        assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    np.testing.assert_array_equal(d_lens.cpu().numpy(), lens)
    assert int(d_nf) == nf


def test_store_keeps_the_sign_of_zero(cuda):
    # -0.0 has code 8 wherever it stands: beside numbers, in a group of zeros, under a saturated
    # scale; numbers that underflow keep their sign too.
    x = torch.zeros(5, 2, 64)
    x[:, 0] = -0.0
    x[:, 1, ::2] = -0.0
    x[0, :, 3], x[0, :, 20] = 6.0, -1.5
    x[1, :, 7] = float("-inf")
    x[2, :, 9], x[2, :, 41] = 3e38, -3e38
    x[3, :, 1], x[3, :, 2] = -1e-38, 1e-38
    x[4, 1, 16:32] = 5000.0
    x = x.bfloat16()
    for kv_scale in (1.0, KVS, 1e-25, 1e25):
        host = np.zeros((1, 2, 16, 36), np.uint8)
        fp4.store(x.double().numpy(), host, np.arange(5), kv_scale)
        k = torch.zeros(1, 2, 16, 36, dtype=torch.uint8, device=cuda)
        v = torch.zeros_like(k)
        slots = torch.arange(5, dtype=torch.int32, device=cuda)
        pa.pa_store_kvcache_fp4(x.to(cuda), x.to(cuda), k, v, slots, kv_scale)
        np.testing.assert_array_equal(k.cpu().numpy(), host)
        assert torch.equal(k, v) and host[0, 0, 4, 0] == 0x88
        key, _ = pa.pa_gather_kvcache_fp4(k, v, slots, kv_scale)
        rows = np.moveaxis(host[0, :, :5], 0, 1)
        want = torch.from_numpy(fp4.expand(rows, kv_scale).astype(np.float32)).bfloat16()
        assert torch.equal(key.cpu().view(torch.int16), want.view(torch.int16))


def test_decode_stores_the_sign_of_zero(cuda):
    # The stores inside the decode: a sequence's last key, and a row that no position owns.
    c = Case(cuda, [40, 0], [1, 1], 8, 2, 128, seed=36)
    c.key[:, :, ::3], c.value[:, :, 1::3] = -0.0, -0.0
    x, new = c.device(), c.new_tokens()
    x["seq_lens"][1] = 0
    c.decode(**x, **new)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_SLOT_MISMATCH
    c.store()
    np.testing.assert_array_equal(x["k_cache"].cpu().numpy(), c.kc)
    np.testing.assert_array_equal(x["v_cache"].cpu().numpy(), c.vc)


@pytest.mark.parametrize("new", [[1] * 64, [8] * 60 + [1] * 4])
def test_prefill_allocates_no_scratch_that_it_does_not_use(cuda, new):
    # One or two blocks of queries a sequence never expand their keys beforehand, so a call without a
    # workspace takes no room for them (64 sequences of up to 32768 keys: 8 GiB).
    c = Case(cuda, [300] * 64, new, 8, 8, 128, seed=37)
    x = c.device()
    cu = _t(c.cu, cuda)
    call = lambda **kw: pa.pa_varlen_prefill_fp4(  # noqa: E731
        x["q"], x["k_cache"], x["v_cache"], cu, x["seq_lens"], x["block_table"], max(new), 32768, c.scale, c.kv_scale, **kw)
    c.check(call())
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    out = call()
    assert torch.cuda.max_memory_allocated() - before <= out.nbytes + 2 * pa.pa_decode_fp4_workspace_size(64, 8, 8, 128, 32768)


# ------------------------------------------------------- limits of the variants ---
@pytest.mark.parametrize("lens,heads,kv_heads,dim", [([90] * 1000, 8, 2, 64), ([17, 90] * 320, 18, 2, 128), ([160] * 3, 8, 2, 128),
                                                     ([159, 160, 1], 32, 2, 64), ([161, 7], 8, 2, 128), ([161] * 3, 32, 2, 64)])
def test_decode_at_the_whole_segment_limit(cuda, lens, heads, kv_heads, dim):
    # Up to 160 keys (five units of 32): whole segments, however many (2000 on 1824 warps, 1280 of
    # two n-tiles on 1216); from 161 on pieces and a merge.
    c = Case(cuda, np.array(lens) - 1, [1] * len(lens), heads, kv_heads, dim, seed=len(lens))
    need = pa.pa_decode_fp4_workspace_size(len(lens), heads, kv_heads, dim, max(lens))
    assert (need == 0) == (max(lens) <= 160)
    c.check(c.decode())


@pytest.mark.parametrize("window", [144, 145, 146, 160])
def test_decode_at_the_windows_whole_segment_limit(cuda, window):
    # A window's keys begin inside a 16-key half: with up to 145 of them five units hold them always.
    c = Case(cuda, [300, 304, 319, 1000, 1001, 15], [1] * 6, 8, 2, 128, seed=window)
    need = pa.pa_decode_fp4_workspace_size(6, 8, 2, 128, int(c.lens.max()), window)
    assert (need == 0) == (window <= 145)
    c.check(c.decode(window), window)


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("heads,kv_heads", [(8, 8), (32, 8), (40, 8)])
def test_prefill_at_the_expansion_limit(cuda, heads, kv_heads, dim):
    # The last query length whose keys are expanded in the kernel, and the first expanded beforehand.
    edge = 4 * (128 // (heads // kv_heads))
    for n in (edge, edge + 1):
        c = Case(cuda, [20, 3], [n, 5], heads, kv_heads, dim, seed=n)
        x = c.device()
        most = int(c.lens.max())
        ws = torch.full((pa.pa_varlen_prefill_fp4_workspace_size(2, heads, kv_heads, dim, most, 0, n),), 0xff, dtype=torch.uint8,
                        device=cuda)
        c.check(pa.pa_varlen_prefill_fp4(x["q"], x["k_cache"], x["v_cache"], _t(c.cu, cuda), x["seq_lens"], x["block_table"], n,
                                         most, c.scale, c.kv_scale, workspace=ws))


def test_a_decode_step_with_empty_rows_at_its_end(cuda):
    # A padded batch: rows without a request have no tokens, stand last and give zeros.
    c = Case(cuda, [40, 15, 700, -1, -1], [1] * 5, 8, 2, 128, seed=38)
    table = c.table.copy()
    nb = c.kc.shape[0]
    free = np.setdiff1d(np.arange(nb), table[table >= 0])
    pool = np.zeros(nb, np.int32)
    pool[: len(free)] = free
    bt, lens = _t(table, cuda), _t([40, 15, 700, 0, 0], cuda)
    lens, _, slots, _, _ = pa.pa_prepare_step(lens, _t([1, 1, 1, 0, 0], cuda), bt, _t(pool, cuda), _t([len(free)], cuda), 16, 5,
                                              seq_lens=lens)
    assert slots[3:].tolist() == [-1, -1] and lens.tolist() == [41, 16, 701, 0, 0]
    x = c.device() | {"block_table": bt, "seq_lens": lens}
    key, value = _bf((5, 2, 128), 80), _bf((5, 2, 128), 81)
    out = c.decode(**x, key=key.to(cuda), value=value.to(cuda), slot_mapping=slots)
    c.key, c.value, c.slots, c.table = key, value, slots.cpu().numpy(), bt.cpu().numpy()
    c.store()
    np.testing.assert_array_equal(x["k_cache"].cpu().numpy(), c.kc)
    c.check(out)
    assert (out[3:] == 0).all()


@pytest.mark.parametrize("what", ["decode", "in the kernel", "beforehand"])
def test_queries_beyond_the_f16_range(cuda, what):
    # Where the products are f16 ones a query beyond 65504 is clamped; with keys expanded beforehand
    # (K bf16, as the queries) it is not.  The small scale keeps the scores below 100.
    new = [1, 1] if what == "decode" else [100, 5]
    c = Case(cuda, [300, 40], new, 8, 2, 128, seed=39)
    c.q = (c.q.float() * 5e4).bfloat16()
    assert int((c.q.abs() > 65504).sum()) > 100
    c.scale = 1e-5
    out = c.decode() if what == "decode" else c.prefill(expand=what == "beforehand")
    if what != "beforehand":
        c.q = c.q.double().clamp(-65504, 65504)
    c.check(out)
