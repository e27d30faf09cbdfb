"""The 4-bit step's calls behind kernels that let their dependents start before they have written
what those read: every call sees the finished data."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import paged_kv_attention_03_gb300 as pa
from paged_kv_attention_03_gb300 import builder
from test_gpu_fp4 import Case, _t

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def early_write(cuda, tmp_path_factory):
    """early_write(dst, src): a kernel on the current stream that triggers its dependents, runs for
    200 us and then copies src to dst (int32)."""
    path = str(tmp_path_factory.mktemp("early") / "early_writer.so")
    subprocess.run([builder._nvcc(), *builder.ARCH_FLAGS, "-O2", "-shared", "-Xcompiler", "-fPIC", "-o", path,
                    os.path.join(HERE, "early_writer.cu")], check=True)
    fn = ctypes.CDLL(path).early_write
    fn.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_uint64, ctypes.c_void_p]

    def write(dst, src):
        assert dst.dtype == src.dtype == torch.int32 and dst.numel() == src.numel()
        assert fn(dst.data_ptr(), src.data_ptr(), dst.numel(), 200_000, torch.cuda.current_stream().cuda_stream) == 0

    return write


def _run(step, out, captured):
    """step() five times, or captured once and replayed: a copy of out after each."""
    main = torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    got = []
    with torch.cuda.stream(main):
        step()
        torch.cuda.synchronize()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=main):
                step()
        for _ in range(5):
            out.fill_(float("nan"))
            graph.replay() if captured else step()
            got.append(out.clone())
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("old", [[1, 1], [2500, 3000], [0, 4000], [4000, 0]])
def test_decode_merges_by_the_lengths_that_an_early_trigger_precedes(cuda, early_write, captured, old):
    # Few long sequences: cut into pieces, and the split kernel leaves SMs free for the merge, which
    # must not work from the lengths that were there before.
    c = Case(cuda, [3999, 2000], [1, 1], 8, 2, 128, seed=50)
    x = c.device()
    want = c.decode(**x)
    c.check(want)
    ws = torch.empty(pa.pa_decode_fp4_workspace_size(2, 8, 2, 128, 4000), dtype=torch.uint8, device=cuda)
    out, lens, before = torch.empty_like(x["q"]), torch.empty_like(x["seq_lens"]), _t(old, cuda)

    def step():
        lens.copy_(before)
        early_write(lens, x["seq_lens"])
        c.decode(**{**x, "seq_lens": lens}, out=out, workspace=ws)

    for got in _run(step, out, captured):
        assert torch.equal(got, want)
    assert pa.pa_read_device_error(device=cuda) == 0


@pytest.mark.parametrize("captured", [False, True])
def test_decode_rows_of_a_packed_call_behind_an_early_trigger(cuda, early_write, captured):
    # Single-row sequences of a packed call, alone (the decode is the call's first kernel) and beside
    # a chunk (it follows the prefill kernel): lengths and row offsets both arrive late.
    for new in ([1, 1, 1], [1, 70, 1]):
        c = Case(cuda, [3999, 100, 2000], new, 8, 2, 128, seed=51)
        x = c.device()
        cu = _t(c.cu, cuda)
        args = (max(new), int(c.lens.max()), c.scale, c.kv_scale)
        want = pa.pa_varlen_prefill_fp4(x["q"], x["k_cache"], x["v_cache"], cu, x["seq_lens"], x["block_table"], *args)
        c.check(want)
        ws = torch.empty(pa.pa_varlen_prefill_fp4_workspace_size(3, 8, 2, 128, args[1]), dtype=torch.uint8, device=cuda)
        out = torch.empty_like(want)
        late = torch.zeros(7, dtype=torch.int32, device=cuda)  # lengths, then offsets
        real = torch.cat([x["seq_lens"], cu])
        before = _t([1, 1, 1, 0, 0, 0, 0], cuda)

        def step():
            late.copy_(before)
            early_write(late, real)
            pa.pa_varlen_prefill_fp4(x["q"], x["k_cache"], x["v_cache"], late[3:], late[:3], x["block_table"], *args,
                                     out=out, workspace=ws)

        for got in _run(step, out, captured):
            assert torch.equal(got, want)
        assert pa.pa_read_device_error(device=cuda) == 0


def test_lengths_of_a_prepared_step_reach_the_merge(cuda):
    # pa_prepare_step in two launches right before a decode of few, cut sequences, in place.
    c = Case(cuda, [3999, 2000], [1, 1], 8, 2, 128, seed=52)
    x = c.device()
    want = c.decode(**x)
    free = _t(np.arange(c.kc.shape[0]), cuda)  # (as many places as the pool has blocks)
    for _ in range(5):
        lens = x["seq_lens"] - 1
        pa.pa_prepare_step(lens, torch.ones_like(lens), x["block_table"].clone(), free, _t([4], cuda), 16, 5000,
                           seq_lens=lens)
        assert torch.equal(c.decode(**{**x, "seq_lens": lens}), want)
    assert pa.pa_read_device_error(device=cuda) == 0


@pytest.mark.parametrize("captured", [False, True])
def test_decode_reads_inputs_that_an_early_trigger_precedes(cuda, early_write, captured):
    # Queries, tables and both caches are written while the decode's blocks may be there already.
    c = Case(cuda, [3999, 2000, 40], [1] * 3, 8, 2, 128, seed=53)
    x = c.device()
    want = c.decode(**x)
    c.check(want)
    late = {k: torch.empty_like(v) for k, v in x.items()}
    out = torch.empty_like(x["q"])
    ws = torch.empty(pa.pa_decode_fp4_workspace_size(3, 8, 2, 128, 4000), dtype=torch.uint8, device=cuda)
    for name in ("q", "block_table", "k_cache", "v_cache"):
        def step():
            for k, v in x.items():
                late[k].copy_(v)
            late[name].view(torch.uint8).fill_(0xff)  # NaN queries and scales, entries of -1
            c.decode(**late, out=out, workspace=ws)  # (its loads of the old values)
            early_write(late[name].view(torch.int32).flatten(), x[name].view(torch.int32).flatten())
            c.decode(**late, out=out, workspace=ws)

        for got in _run(step, out, captured):
            assert torch.equal(got, want), name
        assert pa.pa_read_device_error(device=cuda) == (pa.DEVERR_BLOCK_RANGE if name == "block_table" else 0)


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("captured", [False, True])
def test_expansion_reads_what_an_early_trigger_precedes(cuda, early_write, captured, dim):
    # The expansion of a long prefill's keys: caches, table, lengths and offsets written late.
    c = Case(cuda, [300, 0, 50], [200, 300, 33], 8, 2, dim, seed=54)
    x = c.device() | {"cu": _t(c.cu, cuda)}
    late = {k: torch.empty_like(v) for k, v in x.items()}
    out = torch.empty_like(x["q"])
    ws = torch.empty(pa.pa_varlen_prefill_fp4_workspace_size(3, 8, 2, dim, 800), dtype=torch.uint8, device=cuda)

    def call(y):
        pa.pa_varlen_prefill_fp4(y["q"], y["k_cache"], y["v_cache"], y["cu"], y["seq_lens"], y["block_table"], 768, 800, c.scale,
                                 c.kv_scale, out=out, workspace=ws)

    call(x)
    c.check(out)
    want = out.clone()
    for name in ("block_table", "k_cache", "v_cache", "seq_lens", "cu"):
        def step():
            for k, v in x.items():
                late[k].copy_(v)
            late[name].zero_()
            call(late)
            early_write(late[name].view(torch.int32).flatten(), x[name].view(torch.int32).flatten())
            call(late)

        for got in _run(step, out, captured):
            assert torch.equal(got, want), name
        pa.pa_read_device_error(device=cuda)  # (the call with zeros in the place of lengths is flagged)


@pytest.mark.parametrize("dim", [128, 64])
@pytest.mark.parametrize("captured", [False, True])
def test_prefill_reads_the_rows_of_the_decode_before_it(cuda, captured, dim):
    # A decode stores its new tokens and lets the next call in before it writes them; the next call
    # expands a cache with those rows.
    c = Case(cuda, [700, 2047, 15, 64], [1] * 4, 8, 2, dim, seed=55)
    x, new = c.device(), c.new_tokens()
    start = {k: x[k].clone() for k in ("k_cache", "v_cache")}
    first = c.decode(**x, **new)
    c.store()
    # The prefill: the last rows of every sequence, the new token's the last.
    p = Case.__new__(Case)
    p.__dict__ = dict(c.__dict__)
    p.new = np.array([300, 1, 16, 65])
    p.cu = np.concatenate([[0], np.cumsum(p.new)]).astype(np.int32)
    p.q = torch.randn(int(p.cu[-1]), 8, dim, generator=torch.Generator().manual_seed(56)).bfloat16()
    q, cu = p.q.to(cuda), _t(p.cu, cuda)
    out = torch.empty_like(q)
    ws = torch.empty(pa.pa_varlen_prefill_fp4_workspace_size(4, 8, 2, dim, 2048), dtype=torch.uint8, device=cuda)

    def step():
        for k, v in start.items():
            x[k].copy_(v)
        c.decode(**x, **new)
        pa.pa_varlen_prefill_fp4(q, x["k_cache"], x["v_cache"], cu, x["seq_lens"], x["block_table"], 768, 2048, p.scale,
                                 p.kv_scale, out=out, workspace=ws)

    step()
    p.check(out)
    want = out.clone()
    for got in _run(step, out, captured):
        assert torch.equal(got, want)
    assert torch.equal(c.decode(**x), first)
