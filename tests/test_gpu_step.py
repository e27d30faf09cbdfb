"""Block tables, slots and the free list built on the GPU against the oracle's
request-by-request walk: whole numbers, equal bit for bit."""
import numpy as np
import pytest
import torch

import paged_kv_attention_03_gb300 as pa
from oracle import fp4

pytestmark = pytest.mark.gpu


def _t(a, dev):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32, device=dev)


def _state(ctx, bs, mb, extra, seed):
    """Tables holding the cached tokens' blocks and a shuffled free list of `extra` blocks."""
    rng = np.random.default_rng(seed)
    have = [-(-int(c) // bs) for c in ctx]
    nb = sum(have) + extra
    perm = rng.permutation(nb)
    table = np.full((len(ctx), mb), -7, np.int32)  # entries that nobody may touch
    at = 0
    for i, n in enumerate(have):
        table[i, :n] = perm[at:at + n]
        at += n
    free = np.full(nb, -9, np.int32)
    free[:extra] = perm[at:]
    return table, free, extra


def _check(dev, ctx, q, bs, mb, extra, max_tokens, seed=0, flags=0):
    table, free, nf = _state(ctx, bs, mb, extra, seed)
    want = fp4.prepare_step(ctx, q, table, free, nf, bs, max_tokens)
    bt = _t(table, dev)
    got = pa.pa_prepare_step(_t(ctx, dev), _t(q, dev), bt, _t(free, dev), _t([nf], dev), bs, max_tokens)
    assert pa.pa_read_device_error(device=dev) == flags
    for name, g, w in zip(("seq_lens", "cu_seqlens_q", "slot_mapping", "positions"), got, want[1:]):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    assert int(got[4]) == want[5]
    np.testing.assert_array_equal(bt.cpu().numpy(), want[0])


@pytest.mark.parametrize("bs", [1, 16, 64, 1024])
@pytest.mark.parametrize("ctx,q", [([0], [1]), ([5], [0]), ([0, 0, 0], [0, 0, 0]), ([15, 16, 17], [1, 1, 1]),
                                   ([0, 31, 100, 7, 64], [130, 1, 0, 33, 64]), ([0] * 9, [0, 0, 3, 0, 0, 0, 2, 0, 0])])
def test_prepare_small(cuda, bs, ctx, q):
    mb = max(-(-(c + n) // bs) for c, n in zip(ctx, q)) + 2
    need = sum(-(-(c + n) // bs) + (-c // bs) for c, n in zip(ctx, q))
    for pad in (0, 5):
        _check(cuda, ctx, q, bs, mb, need + 3, sum(q) + pad)


@pytest.mark.parametrize("n,high,bs", [(1, 20000, 16), (33, 700, 16), (700, 40, 32), (5000, 3, 16),
                                       (16384, 2, 64), (64, 1, 16), (600, 90, 1)])
def test_prepare_many(cuda, n, high, bs):
    # One block or two launches, one request or the most there may be.
    rng = np.random.default_rng(n)
    ctx = rng.integers(0, 200, n)
    q = rng.integers(0, high + 1, n)
    q[rng.random(n) < 0.2] = 0
    mb = -(-(200 + high) // bs) + 1
    need = int(sum(-(-(ctx + q) // bs) - -(-ctx // bs)))
    _check(cuda, ctx, q, bs, mb, need, int(q.sum()) + 13, seed=n)


def test_prepare_no_requests(cuda):
    z = torch.zeros(0, dtype=torch.int32, device=cuda)
    got = pa.pa_prepare_step(z, z, torch.zeros(0, 4, dtype=torch.int32, device=cuda), _t([3, 1], cuda),
                             _t([2], cuda), 16, 5)
    assert got[1].tolist() == [0] and got[2].tolist() == [-1] * 5 and got[3].tolist() == [0] * 5
    assert got[4].tolist() == [2] and pa.pa_read_device_error(device=cuda) == 0


@pytest.mark.parametrize("tokens", [6, 9000])
def test_prepare_without_positions(cuda, tokens):
    # The C entry point takes NULL for them.
    ctx, q, bt, free, nf = _t([3, 0], cuda), _t([1, 5], cuda), _t([[7, -1], [-1, -1]], cuda), _t([5, 6], cuda), _t([2], cuda)
    lens, cu, slots = _t([0, 0], cuda), _t([0, 0, 0], cuda), torch.zeros(tokens, dtype=torch.int32, device=cuda)
    p = lambda t: t.data_ptr()  # noqa: E731
    st = pa.load().pa_prepare_step(p(bt), p(lens), p(cu), p(slots), None, p(nf), p(ctx), p(q), p(free), p(nf), 2, 2, tokens, 8,
                                   16, torch.cuda.current_stream().cuda_stream)
    assert st == pa.PA_OK
    assert slots[:6].tolist() == [7 * 16 + 3] + [6 * 16 + i for i in range(5)] and (slots[6:] == -1).all()
    assert lens.tolist() == [4, 5] and nf.tolist() == [1] and pa.pa_read_device_error(device=cuda) == 0


def test_binding_names_what_is_wrong(cuda):
    i = _t([1, 2], cuda)
    table = _t([[0], [0]], cuda)
    with pytest.raises(TypeError, match="query_lens"):
        pa.pa_prepare_step(i, i.long(), table, i, i[:1], 16, 4)
    with pytest.raises(ValueError, match="num_free"):
        pa.pa_prepare_step(i, i, table, i, i, 16, 4)
    with pytest.raises(ValueError, match="slot_mapping"):
        pa.pa_prepare_step(i, i, table, i, i[:1], 16, 4, slot_mapping=i)
    with pytest.raises(ValueError, match="finished"):
        pa.pa_release_blocks(i.cpu(), i, table, i, i[:1], 16)
    with pytest.raises(ValueError, match="contiguous"):
        pa.pa_release_blocks(i, i, _t([[0, 0], [0, 0]], cuda)[:, :1], i, i[:1], 16)


@pytest.mark.parametrize("max_tokens", [200, 20000])
@pytest.mark.parametrize("extra", [0, 1, 4, 7])
def test_prepare_out_of_blocks(cuda, extra, max_tokens):
    # The blocks that are left go to the first requests; the others end with what they hold.
    _check(cuda, [10, 0, 40, 3], [40, 50, 20, 9], 16, 8, extra, max_tokens, flags=pa.DEVERR_NO_BLOCKS)


def test_prepare_clamps_bad_lengths(cuda):
    # Negative lengths count as none; a row's end cuts a request; more tokens than the capacity.
    bt = torch.full((3, 2), -1, dtype=torch.int32, device=cuda)
    free = torch.arange(50, dtype=torch.int32, device=cuda)
    args = (bt, free, _t([50], cuda), 16)
    lens, cu, slots, pos, nf = pa.pa_prepare_step(_t([-3, 0, 0], cuda), _t([2, -1, 40], cuda), *args, 42)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_SEQ_RANGE | pa.DEVERR_QUERY_LEN
    assert lens.tolist() == [2, 0, 32] and cu.tolist() == [0, 2, 2, 42] and nf.tolist() == [47]
    assert slots.tolist() == [49 * 16, 49 * 16 + 1] + [48 * 16 + i for i in range(16)] + \
        [47 * 16 + i for i in range(16)] + [-1] * 8
    assert bt.tolist() == [[49, -1], [-1, -1], [48, 47]]
    lens, cu, slots, pos, nf = pa.pa_prepare_step(_t([0, 0, 0], cuda), _t([6, 6, 6], cuda), *args, 10)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_QUERY_LEN
    assert cu.tolist() == [0, 6, 10, 10] and len(slots) == 10


@pytest.mark.parametrize("n,high,max_tokens", [(3, 9, 0), (3, 40, 10), (40, 60, 5), (40, 200, 3000), (5000, 3, 100),
                                               (16384, 3, 6000), (200, 300, 2048)])
def test_prepare_cuts_at_max_tokens(cuda, n, high, max_tokens):
    # Tokens beyond the capacity are nobody's: no length, table entry or free block counts them.
    rng = np.random.default_rng(n + max_tokens)
    ctx, q = rng.integers(0, 100, n), rng.integers(1, high + 1, n)
    end = np.minimum(np.cumsum(q), max_tokens)
    cut = np.diff(end, prepend=0)
    assert cut.sum() == max_tokens < q.sum()
    table, free, nf = _state(ctx, 16, 30, 6000, 1)
    want = fp4.prepare_step(ctx, cut, table, free, nf, 16, max_tokens)
    bt = _t(table, cuda)
    got = pa.pa_prepare_step(_t(ctx, cuda), _t(q, cuda), bt, _t(free, cuda), _t([nf], cuda), 16, max_tokens)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_QUERY_LEN
    for name, g, w in zip(("seq_lens", "cu_seqlens_q", "slot_mapping", "positions"), got, want[1:]):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
    assert int(got[4]) == want[5]
    np.testing.assert_array_equal(bt.cpu().numpy(), want[0])


def test_prepare_sums_beyond_32_bits(cuda):
    # Lengths whose sum passes 2^32, cut at the capacity; each is cut at its row as well.
    bt = _t([[-1, -1], [60, 61], [-1, -1], [62, -1]], cuda)
    free = torch.arange(70, dtype=torch.int32, device=cuda)
    big = 2**31 - 1
    lens, cu, slots, pos, nf = pa.pa_prepare_step(
        _t([0, 20, 0, 5], cuda), _t([3, big, big, big], cuda), bt, free, _t([50], cuda), 16, 40)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_SEQ_RANGE | pa.DEVERR_QUERY_LEN
    assert lens.tolist() == [3, 32, 0, 5] and cu.tolist() == [0, 3, 40, 40, 40] and nf.tolist() == [49]
    assert slots.tolist() == [49 * 16 + i for i in range(3)] + [61 * 16 + i for i in range(4, 16)] + [-1] * 25
    assert pos.tolist() == [0, 1, 2] + list(range(20, 57))


def test_prepare_flags_bad_block_ids(cuda):
    # A bad id in the free list or in the table gives no slot, and no access.
    bt = torch.tensor([[99, -1], [-1, -1]], dtype=torch.int32, device=cuda)
    free = torch.tensor([1, -5, 1000], dtype=torch.int32, device=cuda)
    _, _, slots, _, nf = pa.pa_prepare_step(_t([3, 0], cuda), _t([1, 17], cuda), bt, free, _t([2], cuda), 16, 18)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE
    assert slots.tolist() == [-1] + [-1] * 16 + [16] and nf.tolist() == [0]
    pa.pa_prepare_step(_t([3, 0], cuda), _t([0, 0], cuda), bt, free, _t([9], cuda), 16, 1)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE  # a count above the pool


@pytest.mark.parametrize("n,high,share,bs", [(1, 50, 1.0, 16), (64, 4096, 0.2, 16), (700, 3000, 0.5, 16),
                                             (3, 20, 0.0, 32), (300, 5, 1.0, 1), (16384, 40, 0.7, 16)])
def test_release(cuda, n, high, share, bs):
    rng = np.random.default_rng(n)
    lens = rng.integers(0, high + 1, n)
    table, free, nf = _state(lens, bs, -(-high // bs) + 1, 11, n)
    fin = (rng.random(n) < share).astype(np.int32) * 5
    want = fp4.release_blocks(fin, lens, table, free, nf, bs)
    f, bt = _t(free, cuda), _t(table, cuda)
    out, count = pa.pa_release_blocks(_t(fin, cuda), _t(lens, cuda), bt, f, _t([nf], cuda), bs)
    assert pa.pa_read_device_error(device=cuda) == 0
    np.testing.assert_array_equal(f.cpu().numpy(), want[0])
    np.testing.assert_array_equal(out.cpu().numpy(), want[1])
    assert int(count) == want[2]
    np.testing.assert_array_equal(bt.cpu().numpy(), table)


@pytest.mark.parametrize("n", [3, 2000])
def test_release_flags_bad_entries(cuda, n):
    # More blocks than the pool has ids, and an id out of range: flagged, nothing written behind.
    lens = torch.full((n,), 32 * 16, dtype=torch.int32, device=cuda)
    bt = torch.zeros(n, 32, dtype=torch.int32, device=cuda)
    buf = torch.full((40,), -3, dtype=torch.int32, device=cuda)
    free = buf[:20]
    _, count = pa.pa_release_blocks(torch.ones_like(lens), lens, bt, free, _t([4], cuda), 16)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE
    assert count.tolist() == [20] and (buf[20:] == -3).all() and (buf[:4] == -3).all()


@pytest.mark.parametrize("n,chunk", [(5, 3), (300, 90)])
def test_steps_in_place_as_a_graph(cuda, n, chunk):
    # Prefill, then decode steps from one captured graph that updates lengths and the free count
    # in place, then releases; the oracle walks along.
    bs, mb = 16, 12
    rng = np.random.default_rng(n)
    table, free, nf = _state([0] * n, bs, mb, n * mb, 1)
    q = rng.integers(1, chunk + 1, n)
    lens, bt, f, count = _t([0] * n, cuda), _t(table, cuda), _t(free, cuda), _t([nf], cuda)
    pa.pa_prepare_step(lens, _t(q, cuda), bt, f, count, bs, n * chunk, seq_lens=lens, num_free_out=count)
    table, want_lens, *_, nf = fp4.prepare_step([0] * n, q, table, free, nf, bs, n * chunk)
    one = torch.ones_like(lens)
    bufs = dict(cu_seqlens_q=torch.empty(n + 1, dtype=torch.int32, device=cuda),
                slot_mapping=torch.empty(n, dtype=torch.int32, device=cuda),
                positions=torch.empty(n, dtype=torch.int32, device=cuda))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_prepare_step(lens, one, bt, f, count, bs, n, seq_lens=lens, num_free_out=count, **bufs)
    for _ in range(40):
        graph.replay()
        table, want_lens, cu, slots, pos, nf = fp4.prepare_step(want_lens, [1] * n, table, free, nf, bs, n)
        for k, w in (("cu_seqlens_q", cu), ("slot_mapping", slots), ("positions", pos)):
            np.testing.assert_array_equal(bufs[k].cpu().numpy(), w)
    np.testing.assert_array_equal(lens.cpu().numpy(), want_lens)
    np.testing.assert_array_equal(bt.cpu().numpy(), table)
    fin = (rng.random(n) < 0.5).astype(np.int32)
    free_np = f.cpu().numpy()
    pa.pa_release_blocks(_t(fin, cuda), lens, bt, f, count, bs, seq_lens_out=lens, num_free_out=count)
    free_np, want_lens, nf = fp4.release_blocks(fin, want_lens, table, free_np, nf, bs)
    np.testing.assert_array_equal(f.cpu().numpy(), free_np)
    np.testing.assert_array_equal(lens.cpu().numpy(), want_lens)
    assert int(count) == nf and pa.pa_read_device_error(device=cuda) == 0
    held = np.concatenate([table[i, : -(-int(c) // bs)] for i, c in enumerate(want_lens)])
    assert sorted([*held, *free_np[:nf]]) == list(range(n * mb))  # every block is somewhere, once


@pytest.mark.parametrize("n,width,extra", [(3, 8, 0), (40, 50, 700), (700, 40, 2), (2000, 64, 0)])
def test_release_keeps_bad_entries_off_the_free_list(cuda, n, width, extra):
    # Rows with -1 and ids past the pool among their blocks, in one launch and in two: flagged, and
    # the list and the count hold the others, in order.  What is left over is sound for a later step.
    rng = np.random.default_rng(n)
    nb = n * width + extra
    table = rng.permutation(nb)[: n * width].reshape(n, width)
    bad = rng.random(table.shape) < 0.1
    bad[0, 0] = bad[n - 1, width - 1] = True
    table = np.where(bad, rng.choice([-1, -2**31, nb, 2**31 - 1], table.shape), table)
    lens = rng.integers(0, width * 16 + 1, n)
    lens[0] = lens[n - 1] = width * 16
    fin = rng.random(n) < 0.7
    fin[0] = fin[n - 1] = True
    held = np.concatenate([table[i, : -(-lens[i] // 16)] for i in range(n) if fin[i]])
    held = held[(held >= 0) & (held < nb)]
    for _ in range(2):  # (the second time with the fault on record)
        free = torch.full((nb,), -9, dtype=torch.int32, device=cuda)
        first = rng.integers(0, nb - len(held) + 1)
        ids = rng.integers(0, nb, first)
        free[:first] = _t(ids, cuda)
        out, count = pa.pa_release_blocks(_t(fin, cuda), _t(lens, cuda), _t(table, cuda), free, _t([first], cuda), 16)
        assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE
        assert int(count) == first + len(held)
        np.testing.assert_array_equal(free[: int(count)].cpu().numpy(), np.concatenate([ids, held]))
        np.testing.assert_array_equal(out.cpu().numpy(), np.where(fin, 0, lens))
    # A release without a fault, behind one with it.
    good = _t(np.arange(n * width).reshape(n, width), cuda)
    free = torch.full((nb,), -9, dtype=torch.int32, device=cuda)
    _, count = pa.pa_release_blocks(_t([1] * n, cuda), _t([width * 16] * n, cuda), good, free, _t([0], cuda), 16)
    assert pa.pa_read_device_error(device=cuda) == 0
    assert int(count) == n * width and torch.equal(free[: n * width], good.flatten())


@pytest.mark.parametrize("n", [4, 500])
def test_release_of_bad_entries_into_a_nearly_full_pool(cuda, n):
    # Valid ids take the places that bad entries before them leave; those beyond the pool are dropped.
    width, nb = 16, n * 16
    table = np.arange(nb).reshape(n, width)
    table[:, ::2] = -1
    lens = np.full(n, width * 16)
    valid = table[table >= 0]
    for room in (len(valid) + 3, len(valid), len(valid) - 5):
        buf = torch.full((nb + 9,), -3, dtype=torch.int32, device=cuda)
        free = buf[:nb]
        start = nb - room
        _, count = pa.pa_release_blocks(_t([1] * n, cuda), _t(lens, cuda), _t(table, cuda), free, _t([start], cuda), 16)
        assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE
        want = valid[:room]
        assert int(count) == start + len(want) and (buf[nb:] == -3).all() and (buf[:start] == -3).all()
        np.testing.assert_array_equal(free[start: int(count)].cpu().numpy(), want)


def test_release_of_a_preempted_row(cuda):
    # A request that got no block has -1 in its table; released by its uncut length, later steps
    # still take sound blocks only.
    bt, free, nf = _t([[-1, -1], [-1, -1]], cuda), _t([5, 4, 3, 2, 1, 0], cuda), _t([2], cuda)
    lens, _, slots, _, nf = pa.pa_prepare_step(_t([0, 0], cuda), _t([17, 20], cuda), bt, free, nf, 16, 37)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_NO_BLOCKS
    assert bt.tolist() == [[4, 5], [-1, -1]] and nf.tolist() == [0]
    _, nf = pa.pa_release_blocks(_t([1, 1], cuda), _t([17, 20], cuda), bt, free, nf, 16)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE
    assert nf.tolist() == [2] and free[:2].tolist() == [4, 5]
    lens, _, slots, _, nf = pa.pa_prepare_step(_t([0, 0], cuda), _t([17, 20], cuda), bt, free, nf, 16, 37)
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_NO_BLOCKS
    assert lens.tolist() == [17, 0] and bt.tolist() == [[5, 4], [-1, -1]] and (slots[:17] >= 0).all()


def test_release_replayed_with_and_without_bad_entries(cuda):
    # A captured release in two launches, replayed over sound rows, rows with bad entries and sound
    # ones again, while another stream releases rows with bad entries all the time.
    n, width = 300, 40
    nb = n * width
    sound = np.arange(nb).reshape(n, width)
    broken = np.where(np.random.default_rng(3).random(sound.shape) < 0.2, -1, sound)
    table, lens, one = _t(sound, cuda), _t([width * 16] * n, cuda), _t([1] * n, cuda)
    free, count, out = (torch.empty(k, dtype=torch.int32, device=cuda) for k in (nb, 1, n))
    zero = _t([0], cuda)
    other = [_t(broken, cuda), torch.empty(nb, dtype=torch.int32, device=cuda), torch.empty(n, dtype=torch.int32, device=cuda),
             torch.empty(1, dtype=torch.int32, device=cuda)]
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(main):
        pa.pa_release_blocks(one, lens, table, free, zero, 16, seq_lens_out=out, num_free_out=count)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=main):
            pa.pa_release_blocks(one, lens, table, free, zero, 16, seq_lens_out=out, num_free_out=count)
    for rows in (sound, broken, sound, broken):
        want = rows[rows >= 0]
        with torch.cuda.stream(main):
            table.copy_(_t(rows, cuda))
            free.fill_(-9)
        torch.cuda.synchronize()
        for _ in range(5):
            with torch.cuda.stream(side):
                pa.pa_release_blocks(one, lens, other[0], other[1], zero, 16, seq_lens_out=other[2], num_free_out=other[3])
            with torch.cuda.stream(main):
                graph.replay()
        torch.cuda.synchronize()
        assert int(count) == len(want) and int(other[3]) == (broken >= 0).sum()
        np.testing.assert_array_equal(free[: len(want)].cpu().numpy(), want)
        np.testing.assert_array_equal(other[1][: int(other[3])].cpu().numpy(), broken[broken >= 0])
    assert pa.pa_read_device_error(device=cuda) == pa.DEVERR_BLOCK_RANGE
