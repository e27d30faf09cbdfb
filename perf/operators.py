"""What is measured of the serving step over a 4-bit KV cache, and the plain form of each operator.

The operators, in the order a serving step runs them:

* ``prepare``: block tables, slot mapping, positions and lengths of a step, built on the GPU from the requests' lengths and
  a free list of blocks (``pa_prepare_step``);
* ``release``: the blocks of finished requests go back to the free list (``pa_release_blocks``);
* ``store``: new K/V rows are quantised into the 4-bit cache and read back (``pa_store_kvcache_fp4``, ``pa_gather_kvcache_fp4``);
* ``prefill``: packed variable-length causal attention over the 4-bit cache (``pa_varlen_prefill_fp4``);
* ``decode``: one query per sequence over the 4-bit cache (``pa_decode_fp4``).

The cache: ``[num_blocks, num_kv_heads, block_size, head_dim / 2 + head_dim / 16]`` bytes.  A row holds the E2M1 codes of one
token and kv head, two to a byte (even dimension in the low four bits), then one E4M3 scale for each 16 dimensions; an element
is code * scale * kv_scale.
"""
import numpy as np
import torch

own = False

E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # The metadata of one decode step of 64 requests (the batched decode workload): latency.
        {"name": "prepare decode step", "op": "prepare", "chunks": 0, "chunk_low": 1, "chunk_high": 1, "decodes": 64,
         "ctx_low": 511, "ctx_high": 4095, "block": 16},
        # A large mixed step: ragged prompts and chunks beside many decodes, pages of 32.
        {"name": "prepare mixed step", "op": "prepare", "chunks": 256, "chunk_low": 1, "chunk_high": 2048, "decodes": 1777,
         "ctx_low": 0, "ctx_high": 8192, "block": 32},
        # A few of a batch's requests end.
        {"name": "release few", "op": "release", "requests": 64, "share": 0.15, "low": 512, "high": 4096, "block": 16},
        # A large batch is cleared by half, long contexts.
        {"name": "release many", "op": "release", "requests": 1024, "share": 0.5, "low": 1, "high": 16384, "block": 16},
        # The new tokens of one decode step.
        {"name": "store decode step", "op": "store", "tokens": 64, "kv_heads": 8, "dim": 128, "block": 16, "padding": 0.1},
        # The tokens of a prefill step, a ragged number of them.
        {"name": "store prefill step", "op": "store", "tokens": 17403, "kv_heads": 8, "dim": 128, "block": 16, "padding": 0.02},
        # The smallest decode: four short sequences, 8/2 heads of 64 (latency).
        {"name": "decode tiny", "op": "decode", "batch": 4, "heads": 8, "kv_heads": 2, "dim": 64, "block": 16, "low": 17,
         "high": 100, "window": 0},
        # The batched decode workload: 64 requests of 512 to 4096 keys, 32/8 heads.
        {"name": "decode batched", "op": "decode", "batch": 64, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16,
         "low": 512, "high": 4096, "window": 0},
        # The long decode workload: 8 requests of 32k to 131k keys, 40/8 heads.
        {"name": "decode long", "op": "decode", "batch": 8, "heads": 40, "kv_heads": 8, "dim": 128, "block": 16,
         "low": 32768, "high": 131072, "window": 0},
        # A few short prompts with a cached context, odd lengths, pages of 64.
        {"name": "prefill few chunks", "op": "prefill", "prompts": 3, "low": 37, "high": 301, "ctx_low": 0, "ctx_high": 700,
         "decodes": 0, "heads": 32, "kv_heads": 8, "dim": 128, "block": 64, "window": 0},
        # The varlen prefill workload: 16 prompts of 128 to 2048 tokens.
        {"name": "prefill varlen", "op": "prefill", "prompts": 16, "low": 128, "high": 2048, "ctx_low": 0, "ctx_high": 0,
         "decodes": 0, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "window": 0},
        # Chunked prefill beside decodes in one call, with a sliding window.
        {"name": "prefill mixed window", "op": "prefill", "prompts": 4, "low": 512, "high": 512, "ctx_low": 1024,
         "ctx_high": 4096, "decodes": 24, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "window": 2048},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return int(round(float(low) * (float(high) / low) ** rng.random()))


def draw(rng):
    op = rng.choice(("prepare", "release", "store", "decode", "decode", "prefill", "prefill"))
    block = rng.choice((16, 32, 64))
    if op == "prepare":
        chunk = _spread(rng, 1, 2048)
        return {"op": op, "chunks": _spread(rng, 1, 257) - 1, "chunk_low": 1 + chunk // rng.randint(2, 9), "chunk_high": chunk + 1,
                "decodes": _spread(rng, 1, 1800), "ctx_low": rng.randint(0, 40), "ctx_high": _spread(rng, 41, 8192), "block": block}
    if op == "release":
        return {"op": op, "requests": _spread(rng, 1, 1024), "share": round(rng.random(), 3), "low": rng.randint(1, 40),
                "high": _spread(rng, 41, 16384), "block": block}
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    if op == "store":
        return {"op": op, "tokens": _spread(rng, 1, 17403), "kv_heads": kv_heads, "dim": dim, "block": block,
                "padding": round(0.3 * rng.random(), 3)}
    heads = kv_heads * rng.choice((1, 2, 4, 5, 7, 8, 16))
    if heads > 40:
        heads = kv_heads * 5
    if op == "decode":
        high = _spread(rng, 30, 60000)
        batch = _spread(rng, 1, max(2, min(700, 8 * 131072 * 8 // (2 * high * kv_heads))))
        return {"op": op, "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim, "block": block,
                "low": 1 + high // rng.randint(2, 20), "high": high, "window": rng.choice((0, 0, 1 + rng.randint(1, high)))}
    high = _spread(rng, 3, 1500)
    ctx = rng.choice((0, _spread(rng, 1, 2000)))
    prompts = _spread(rng, 1, max(2, min(100, int(16 * 32 * 2048 * 2048 // (2 * heads * high * (high + ctx))))))
    decodes = rng.choice((0, rng.randint(1, 9))) if prompts < 16 else 0
    return {"op": op, "prompts": prompts, "low": 1 + high // rng.randint(2, 9), "high": high, "ctx_low": ctx // 2, "ctx_high": ctx,
            "decodes": decodes, "heads": min(heads, 32 // kv_heads * kv_heads), "kv_heads": kv_heads, "dim": dim, "block": block,
            "window": rng.choice((0, 0, 1 + rng.randint(1, high + ctx)))}


# ------------------------------------------------------ the 4-bit cache, plainly ---
def _quantise(x, kv_scale):
    """Rows [..., dim] as the cache's bytes [..., dim / 2 + dim / 16].  Every division is one in 32 bits: the scale of 16
    elements is E4M3(max|x| / (6 kv_scale)), at least the smallest E4M3 number, and a code E2M1(x / (scale kv_scale)), both
    to the nearest, ties to even, saturating."""
    x = x.float().unflatten(-1, (-1, 16))
    six = torch.tensor(6.0 * float(np.float32(kv_scale)), dtype=torch.float32, device=x.device)
    one = torch.tensor(kv_scale, dtype=torch.float32, device=x.device)
    scale = (x.abs().amax(-1, keepdim=True) / six).clamp(min=2.0 ** -9, max=448.0).to(torch.float8_e4m3fn)
    y = x / (scale.float() * one)
    a = y.abs()
    code = (a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte() + (a > 2.5).byte() \
        + (a >= 3.5).byte() + (a > 5.0).byte() + 8 * torch.signbit(y).byte()
    code = code.flatten(-2)
    return torch.cat([code[..., 0::2] + 16 * code[..., 1::2], scale.squeeze(-1).view(torch.uint8)], dim=-1)


def _values(rows, kv_scale):
    """The numbers that the cache's rows stand for, in 32 bits."""
    dim = rows.shape[-1] * 16 // 9
    codes = rows[..., : dim // 2]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=rows.device)
    v = table[torch.stack([codes & 15, codes >> 4], dim=-1).int()].flatten(-2)
    scale = rows[..., dim // 2:].contiguous().view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (-1, 16)) * scale[..., None]).flatten(-2) * kv_scale


def _cache(num_blocks, kv_heads, block, dim, kv_scale, g):
    """A cache that holds quantised N(0, 1) values everywhere."""
    rows = torch.empty(num_blocks, kv_heads, block, dim // 2 + dim // 16, dtype=torch.uint8, device="cuda")
    slab = max(1, (1 << 26) // (kv_heads * block * dim))
    for s in range(0, num_blocks, slab):
        part = rows[s:s + slab]
        part.copy_(_quantise(torch.randn(*part.shape[:-1], dim, generator=g, device="cuda").bfloat16(), kv_scale))
    return rows


# ---------------------------------------------------------------- inputs ---
def _between(low, high, n, g):
    """n whole numbers between low and high: the same ones for every seed, so that outputs keep their shapes, in the seed's order."""
    n_ = torch.randint(low, high + 1, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int64)
    return n_[torch.randperm(n, generator=g)]


def _tables(blocks, num_blocks, g, width=None):
    """Shuffled distinct blocks for rows of blocks[i] entries, -1 behind them; and the pool's blocks that are left."""
    perm = torch.randperm(num_blocks, generator=g, dtype=torch.int64)
    col = torch.arange(width or max(int(blocks.max()), 1))
    first = blocks.cumsum(0) - blocks
    at = (first[:, None] + col).clamp(max=num_blocks - 1)
    return torch.where(col < blocks[:, None], perm[at], -1), perm[int(blocks.sum()):]


def _lengths(case, g):
    """(cached, new) tokens of each request of a prepare or prefill case, the decodes behind the chunks."""
    n = case["chunks"] if case["op"] == "prepare" else case["prompts"]
    low, high = (case["chunk_low"], case["chunk_high"]) if case["op"] == "prepare" else (case["low"], case["high"])
    new = torch.cat([_between(low, high, n, g), torch.ones(case["decodes"], dtype=torch.int64)])
    return _between(case["ctx_low"], case["ctx_high"], n + case["decodes"], g), new


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    d = torch.Generator(device="cuda").manual_seed(seed + 1)
    dev = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    bs = case["block"]
    s = {"case": case}
    if case["op"] == "prepare":
        ctx, new = _lengths(case, g)
        have = (ctx + bs - 1) // bs
        most = (case["ctx_high"] + case["chunk_high"] + bs) // bs  # blocks of a request
        num_blocks = most * len(ctx) + 64
        table, left = _tables(have, num_blocks, g, most + 3)
        free = torch.zeros(num_blocks, dtype=torch.int64)
        free[: len(left)] = left
        tokens = case["chunks"] * case["chunk_high"] + case["decodes"]  # the capacity that a captured step is built for
        n = len(ctx)
        s |= {"context_lens": dev(ctx), "query_lens": dev(new), "block_table": dev(table), "free_blocks": dev(free),
              "num_free": dev(torch.tensor([len(left)])), "max_tokens": tokens,
              "out": {k: torch.empty(m, dtype=torch.int32, device="cuda") for k, m in
                      (("seq_lens", n), ("cu_seqlens_q", n + 1), ("slot_mapping", tokens), ("positions", tokens), ("num_free_out", 1))}}
        return s
    if case["op"] == "release":
        lens = _between(case["low"], case["high"], case["requests"], g)
        blocks = (lens + bs - 1) // bs
        num_blocks = int(blocks.sum()) + 64
        table, left = _tables(blocks, num_blocks, g)
        free = torch.zeros(num_blocks, dtype=torch.int64)
        free[: len(left)] = left
        s |= {"finished": dev(torch.rand(len(lens), generator=g) < case["share"]), "seq_lens": dev(lens), "block_table": dev(table),
              "free_blocks": dev(free), "num_free": dev(torch.tensor([len(left)])),
              "out": {"seq_lens_out": torch.empty(len(lens), dtype=torch.int32, device="cuda"),
                      "num_free_out": torch.empty(1, dtype=torch.int32, device="cuda")}}
        return s
    hkv, dim = case["kv_heads"], case["dim"]
    s["kv_scale"] = 0.7
    if case["op"] == "store":
        t = case["tokens"]
        num_blocks = (t + bs - 1) // bs + 9
        slots = torch.randperm(num_blocks * bs, generator=g)[:t]
        slots[torch.rand(t, generator=g) < case["padding"]] = -1
        size = torch.exp(torch.randn(t, hkv, 1, generator=d, device="cuda"))  # tokens and heads differ in magnitude
        s |= {"slot_mapping": dev(slots),
              "key": (size * torch.randn(t, hkv, dim, generator=d, device="cuda")).bfloat16(),
              "value": torch.randn(t, hkv, dim, generator=d, device="cuda").bfloat16(),
              "k_cache": torch.zeros(num_blocks, hkv, bs, dim // 2 + dim // 16, dtype=torch.uint8, device="cuda"),
              "v_cache": torch.zeros(num_blocks, hkv, bs, dim // 2 + dim // 16, dtype=torch.uint8, device="cuda")}
        s["rows"] = [torch.empty_like(s["key"]), torch.empty_like(s["value"])]
        return s
    if case["op"] == "decode":
        lens = _between(case["low"], case["high"], case["batch"], g)
        new = torch.ones_like(lens)
    else:
        ctx, new = _lengths(case, g)
        lens = ctx + new
    blocks = (lens + bs - 1) // bs
    num_blocks = int(blocks.sum()) + 9
    table, _ = _tables(blocks, num_blocks, g)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    s |= {"lens": lens.tolist(), "new": new.tolist(), "seq_lens": dev(lens), "cu_seqlens_q": dev(cu), "block_table": dev(table),
          "max_seq_len": int(lens.max()), "max_query_len": int(new.max()), "scale": dim ** -0.5,
          "q": torch.randn(int(cu[-1]), case["heads"], dim, generator=d, device="cuda").bfloat16(),
          "k_cache": _cache(num_blocks, hkv, bs, dim, s["kv_scale"], d), "v_cache": _cache(num_blocks, hkv, bs, dim, s["kv_scale"], d)}
    s["o"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------ plain forms ---
def _plain_prepare(s):
    bs, ctx, new = s["case"]["block"], s["context_lens"].long(), s["query_lens"].long()
    table, free, num_free = s["block_table"].long(), s["free_blocks"].long(), s["num_free"].long()
    have, lens = (ctx + bs - 1) // bs, ctx + new
    need = (lens + bs - 1) // bs - have
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0)])
    first = need.cumsum(0) - need
    # The table: blocks have .. have + need - 1 of a row are the next ones from the end of the free list.
    col = torch.arange(table.shape[1], device=table.device)
    rank = first[:, None] + col - have[:, None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    table = torch.where(fresh, free[(num_free - 1 - rank).clamp(0, len(free) - 1)], table)
    # The tokens.
    t = torch.arange(s["max_tokens"], device=table.device)
    seq = torch.searchsorted(cu[1:], t, right=True).clamp(max=len(ctx) - 1)
    pos = ctx[seq] + t - cu[seq]
    used = t < cu[-1]
    pos = torch.where(used, pos, 0)
    slot = torch.where(used, table[seq, (pos // bs).clamp(max=table.shape[1] - 1)] * bs + pos % bs, -1)
    return {"block_table": table.int(), "seq_lens": lens.int(), "cu_seqlens_q": cu.int(), "slot_mapping": slot.int(),
            "positions": pos.int(), "num_free": (num_free - need.sum()).int()}


def _plain_release(s):
    bs, lens, table = s["case"]["block"], s["seq_lens"].long(), s["block_table"].long()
    free, num_free = s["free_blocks"].long(), s["num_free"].long()
    done = s["finished"] != 0
    n = torch.where(done, (lens + bs - 1) // bs, 0)
    last = n.cumsum(0)
    at = torch.arange(len(free), device=free.device) - num_free
    row = torch.searchsorted(last, at, right=True).clamp(max=len(lens) - 1)
    col = (at - (last - n)[row]).clamp(0, table.shape[1] - 1)
    free = torch.where((at >= 0) & (at < last[-1]), table[row, col], free)
    return {"free_blocks": free.int(), "seq_lens": torch.where(done, 0, lens).int(), "num_free": (num_free + last[-1]).int()}


def _plain_store(s):
    bs, slots = s["case"]["block"], s["slot_mapping"].long()
    heads = torch.arange(s["case"]["kv_heads"], device=slots.device)
    # A skipped token (slot -1) writes the bytes that are there already in a place that no token uses: behind the cache.
    got = []
    for x, cache in ((s["key"], s["k_cache"]), (s["value"], s["v_cache"])):
        longer = torch.cat([cache, torch.zeros_like(cache[:1])])
        slot = torch.where(slots < 0, cache.shape[0] * bs, slots)
        longer[(slot // bs)[:, None], heads, (slot % bs)[:, None]] = _quantise(x, s["kv_scale"])
        rows = longer[(slot // bs)[:, None], heads, (slot % bs)[:, None]]
        got.append(torch.where(slots[:, None, None] < 0, 0, _values(rows, s["kv_scale"])).bfloat16())
    return {"key": got[0], "value": got[1]}


def _plain_attention(s):
    """Padded to the longest sequence: gather and expand the cache, scores, mask, softmax, weighted sum, all in 32 bits."""
    case = s["case"]
    bs, hkv, w = case["block"], case["kv_heads"], case["window"]
    cu, lens, table = s["cu_seqlens_q"].long(), s["seq_lens"].long(), s["block_table"].long().clamp(min=0)
    new = cu[1:] - cu[:-1]
    n, most = len(lens), s["max_query_len"]
    row = torch.arange(most, device=cu.device)
    at = (cu[:-1, None] + row).clamp(max=len(s["q"]) - 1)
    q = s["q"].float()[at].unflatten(2, (hkv, -1))  # [n, most, hkv, group, dim]
    group, dim = q.shape[3], q.shape[4]
    q = q.permute(0, 2, 3, 1, 4).reshape(n, hkv, group * most, dim)
    expand = lambda c: _values(c[table], s["kv_scale"]).transpose(1, 2).reshape(n, hkv, -1, dim)  # noqa: E731
    p = ((q @ expand(s["k_cache"]).transpose(2, 3)) * s["scale"]).unflatten(2, (group, most))
    key = torch.arange(p.shape[-1], device=cu.device)
    pos = (lens - new)[:, None] + row  # [n, most]
    see = (key <= pos[..., None]) & (key < lens[:, None, None])
    if w > 0:
        see = see & (key > pos[..., None] - w)
    p = p.masked_fill(~see[:, None, None], float("-inf"))
    p = torch.exp(p - p.amax(-1, keepdim=True).clamp(min=-3e38))
    o = p.flatten(2, 3) @ expand(s["v_cache"])
    o = o / p.sum(-1).flatten(2, 3)[..., None].clamp(min=1e-30)
    o = o.unflatten(2, (group, most)).permute(0, 3, 1, 2, 4).reshape(n, most, hkv * group, dim)
    t = torch.arange(len(s["q"]), device=cu.device)
    seq = torch.searchsorted(cu[1:], t, right=True)
    return o[seq, t - cu[seq]].bfloat16()


def _own(s):
    import paged_kv_attention_03_gb300 as pa
    case = s["case"]
    if case["op"] in ("decode", "prefill") and "workspace" not in s:  # a serving loop keeps it
        size = pa.pa_decode_fp4_workspace_size if case["op"] == "decode" else pa.pa_varlen_prefill_fp4_workspace_size
        need = size(len(s["lens"]), case["heads"], case["kv_heads"], case["dim"], s["max_seq_len"], case["window"])
        s["workspace"] = torch.empty(max(need, 256), dtype=torch.uint8, device="cuda")
    if case["op"] == "prepare":
        pa.pa_prepare_step(s["context_lens"], s["query_lens"], s["block_table"], s["free_blocks"], s["num_free"], case["block"],
                           s["max_tokens"], **s["out"])
        o = s["out"]
        return {"block_table": s["block_table"], "seq_lens": o["seq_lens"], "cu_seqlens_q": o["cu_seqlens_q"],
                "slot_mapping": o["slot_mapping"], "positions": o["positions"], "num_free": o["num_free_out"]}
    if case["op"] == "release":
        o = s["out"]
        pa.pa_release_blocks(s["finished"], s["seq_lens"], s["block_table"], s["free_blocks"], s["num_free"], case["block"], **o)
        return {"free_blocks": s["free_blocks"], "seq_lens": o["seq_lens_out"], "num_free": o["num_free_out"]}
    if case["op"] == "store":
        pa.pa_store_kvcache_fp4(s["key"], s["value"], s["k_cache"], s["v_cache"], s["slot_mapping"], s["kv_scale"])
        key, value = pa.pa_gather_kvcache_fp4(s["k_cache"], s["v_cache"], s["slot_mapping"], s["kv_scale"], key=s["rows"][0],
                                              value=s["rows"][1])
        return {"key": key, "value": value}
    if case["op"] == "decode":
        return pa.pa_decode_fp4(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["max_seq_len"], s["scale"],
                                s["kv_scale"], case["window"], out=s["o"], workspace=s["workspace"])
    return pa.pa_varlen_prefill_fp4(s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens_q"], s["seq_lens"], s["block_table"],
                                    s["max_query_len"], s["max_seq_len"], s["scale"], s["kv_scale"], case["window"], out=s["o"],
                                    workspace=s["workspace"])


def run(s):
    if own:
        return _own(s)
    return {"prepare": _plain_prepare, "release": _plain_release, "store": _plain_store}.get(s["case"]["op"], _plain_attention)(s)


# ------------------------------------------------------------------ work ---
def work(case):
    """Expected bytes and operations: lengths at the middle of their range."""
    bs = case["block"]
    mid = lambda a, b: (a + b) / 2  # noqa: E731
    if case["op"] == "prepare":
        n = case["chunks"] + case["decodes"]
        tokens = case["chunks"] * mid(case["chunk_low"], case["chunk_high"]) + case["decodes"]
        cap = case["chunks"] * case["chunk_high"] + case["decodes"]
        # lengths read, lengths and offsets written; a slot and a position for every token; a free block read and a table
        # entry written for every block's worth of tokens
        return {"bytes": 16 * n + 8 * cap + 8 * tokens / bs, "flops": 0}
    if case["op"] == "release":
        blocks = case["requests"] * case["share"] * mid(case["low"], case["high"]) / bs
        return {"bytes": 12 * case["requests"] + 8 * blocks, "flops": 0}
    hkv, dim = case["kv_heads"], case["dim"]
    row = hkv * (dim // 2 + dim // 16)
    if case["op"] == "store":
        # bf16 rows read, cache rows written; cache rows read, bf16 rows written (K and V)
        return {"bytes": case["tokens"] * 2 * (2 * row + 4 * hkv * dim), "flops": 0}
    if case["op"] == "decode":
        keys = mid(case["low"], case["high"])
        keys = min(keys, case["window"]) if case["window"] > 0 else keys
        pairs = case["batch"] * keys
        return {"bytes": 2 * row * pairs + 4 * case["batch"] * case["heads"] * dim, "flops": 4 * case["heads"] * dim * pairs}
    new, ctx = mid(case["low"], case["high"]), mid(case["ctx_low"], case["ctx_high"])
    w = case["window"] if case["window"] > 0 else 1e18
    pairs = case["prompts"] * new * min(ctx + new / 2, w) + case["decodes"] * min(ctx + 1, w)
    keys = case["prompts"] * min(ctx + new, w + new) + case["decodes"] * min(ctx + 1, w)
    tokens = case["prompts"] * new + case["decodes"]
    return {"bytes": 2 * row * keys + 4 * tokens * case["heads"] * dim, "flops": 4 * case["heads"] * dim * pairs}


# ------------------------------------------------------------- 64 bits ---
def _nearest(x, numbers):
    """The index of the number of an ascending list that is nearest to x; from the middle of two, the even index."""
    v = torch.tensor(numbers, dtype=torch.float64, device=x.device)
    mid = (v[1:] + v[:-1]) / 2
    i = torch.searchsorted(mid, x.contiguous())
    tie = mid[i.clamp(max=len(mid) - 1)] == x
    return i + (tie & (i % 2 == 1))


def _e4m3_numbers():
    return [(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)]


def _exact_store(s):
    scale_numbers = torch.tensor(_e4m3_numbers(), dtype=torch.float64, device="cuda")
    code_numbers = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    kv = np.float32(s["kv_scale"])
    rounded = lambda t: t.to(torch.float32).double()  # noqa: E731  (the definition's divisions and products are 32-bit ones)
    out = []
    for x in (s["key"], s["value"]):
        x = x.double().reshape(-1, 16)
        top = rounded(x.abs().max(dim=1).values / float(np.float32(6) * kv))
        scale = scale_numbers[_nearest(top, _e4m3_numbers()).clamp(min=1)]
        y = rounded(x / rounded(scale * float(kv))[:, None])
        v = code_numbers[_nearest(y.abs(), E2M1)] * torch.sign(x) * scale[:, None] * float(kv)
        v = v.reshape(s["key"].shape)
        v[s["slot_mapping"] < 0] = 0
        out.append(v)
    return {"key": out[0], "value": out[1]}


def _exact_rows(cache, blocks, length, kv_scale, dim):
    """[kv_heads, length, dim] in 64 bits, from the bits of the formats."""
    rows = cache[blocks].transpose(0, 1).flatten(1, 2)[:, :length].int()
    low, high = rows[..., : dim // 2] & 15, rows[..., : dim // 2] >> 4
    c = torch.stack([low, high], dim=-1).flatten(-2)
    e, m = (c >> 1) & 3, (c & 1).double()
    v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.pow(2.0, (e - 1).double())) * (1 - 2 * (c >> 3))
    b = rows[..., dim // 2:]
    e, m = (b >> 3) & 15, (b & 7).double()
    scale = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.pow(2.0, (e - 7).double())) * (1 - 2 * (b >> 7))
    return v * torch.repeat_interleave(scale, 16, dim=-1) * float(np.float32(kv_scale))


def _exact_attention(s):
    case = s["case"]
    bs, hkv, dim, w = case["block"], case["kv_heads"], case["dim"], case["window"]
    group = case["heads"] // hkv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    start = 0
    for i, (length, new) in enumerate(zip(s["lens"], s["new"])):
        blocks = s["block_table"][i, : (length + bs - 1) // bs].long()
        k = _exact_rows(s["k_cache"], blocks, length, s["kv_scale"], dim)
        v = _exact_rows(s["v_cache"], blocks, length, s["kv_scale"], dim)
        q = s["q"][start:start + new].double()
        pos = torch.arange(length - new, length, device="cuda")[:, None]
        key = torch.arange(length, device="cuda")
        hidden = (key > pos) | ((key <= pos - w) if w > 0 else torch.zeros_like(key > pos))
        for h in range(case["heads"]):
            logit = q[:, h] @ k[h // group].T * s["scale"]
            out[start:start + new, h] = torch.softmax(logit.masked_fill(hidden, float("-inf")), dim=-1) @ v[h // group]
        start += new
    return out


def exact(case, seed):
    if case["op"] in ("prepare", "release"):
        return None  # whole numbers: the plain form's are compared as they are
    s = prepare(case, seed)
    return _exact_store(s) if case["op"] == "store" else _exact_attention(s)
