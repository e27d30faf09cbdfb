"""Plain CPU oracle of the 4-bit KV cache and of the step's block tables (numpy, fp64).

TEST INFRASTRUCTURE ONLY, like the rest of this package: it shares no code with the CUDA
library and states each definition directly.

* E2M1: 0, .5, 1, 1.5, 2, 3, 4, 6 with a sign bit; E4M3 ("fn"): no infinities, largest 448.
* A cache row of one token and kv head: D / 2 bytes of codes (even dim in the low four bits),
  then D / 16 scales; element = code * scale * kv_scale.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
# E4M3 values of codes 0 .. 126 (127 is NaN): subnormals m 2^-9, then (1 + m / 8) 2^(e - 7).
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def nearest_code(x: np.ndarray, values: np.ndarray) -> np.ndarray:
    """Code (index into the ascending values) nearest to x >= 0; halfway cases go to the even
    code; values beyond the last one saturate."""
    x = np.asarray(x, np.float64)
    hi = np.clip(np.searchsorted(values, x), 0, len(values) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = x - values[lo], values[hi] - x
    pick_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (x >= values[-1])
    return np.where(pick_hi, hi, lo)


def quantise(x, kv_scale: float) -> np.ndarray:
    """[..., D] float values (bf16 numbers) -> rows [..., D/2 + D/16] uint8."""
    x = np.asarray(x, np.float32)
    d = x.shape[-1]
    kv = np.float32(kv_scale)
    g = x.reshape(*x.shape[:-1], d // 16, 16)
    with np.errstate(all="ignore"):
        top = np.abs(g).max(-1)  # NaN if any is
        scale = np.maximum(nearest_code(np.nan_to_num(top / (np.float32(6) * kv), nan=0.0, posinf=1e9),
                                        E4M3), 1)
        nan = np.isnan(top)
        den = E4M3[scale].astype(np.float32) * kv
        y = g / den[..., None]
        code = nearest_code(np.nan_to_num(np.abs(y), nan=0.0, posinf=1e9), E2M1)
    code = code | np.where(np.signbit(y), 8, 0)
    code = code.reshape(x.shape).astype(np.uint8)
    scale = np.where(nan, 127, scale).astype(np.uint8)
    return np.concatenate([code[..., 0::2] | (code[..., 1::2] << 4), scale], axis=-1)


def expand(rows: np.ndarray, kv_scale: float) -> np.ndarray:
    """Rows [..., D/2 + D/16] uint8 -> [..., D] float64 (NaN where the scale is)."""
    d = rows.shape[-1] // 9 * 16
    c = np.stack([rows[..., : d // 2] & 15, rows[..., : d // 2] >> 4], axis=-1)
    c = c.reshape(*rows.shape[:-1], d)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    s = rows[..., d // 2:].astype(np.int64)
    table = np.concatenate([E4M3, [np.nan]])
    s = np.where(s & 128, -1.0, 1.0) * table[s & 127]
    return v * np.repeat(s, 16, axis=-1) * float(np.float32(kv_scale))


def store(x, cache: np.ndarray, slot_mapping, kv_scale: float) -> None:
    """Quantise rows x [T, Hkv, D] into cache [NB, Hkv, bs, row] in place; slots < 0 and past
    the pool are skipped."""
    nb, _, bs, _ = cache.shape
    rows = quantise(x, kv_scale)
    for t, s in enumerate(np.asarray(slot_mapping)):
        if 0 <= s < nb * bs:
            cache[s // bs, :, s % bs] = rows[t]


def paged_attention(q, k_cache, v_cache, cu_seqlens_q, seq_lens, block_table, num_heads: int,
                    window: int, scale: float, kv_scale: float):
    """Packed attention over 4-bit caches in fp64: (out [Tq, H, D], weight [Tq, H, D]) where
    weight is the same sum over |V| (the size that rounding errors are relative to)."""
    q = np.asarray(q, np.float64)
    bs, hkv = k_cache.shape[2], k_cache.shape[1]
    group = num_heads // hkv
    out = np.zeros(q.shape)
    weight = np.zeros(q.shape)
    for i, length in enumerate(np.asarray(seq_lens)):
        a, b = int(cu_seqlens_q[i]), int(cu_seqlens_q[i + 1])
        if b == a or length == 0:
            continue
        blocks = np.asarray(block_table)[i, : (length + bs - 1) // bs]
        k = expand(k_cache[blocks], kv_scale).transpose(1, 0, 2, 3).reshape(hkv, -1, q.shape[2])[:, :length]
        v = expand(v_cache[blocks], kv_scale).transpose(1, 0, 2, 3).reshape(hkv, -1, q.shape[2])[:, :length]
        pos = length - (b - a) + np.arange(b - a)
        key = np.arange(length)
        see = key[None] <= pos[:, None]
        if window > 0:
            see &= key[None] > pos[:, None] - window
        for h in range(num_heads):
            s = np.where(see, q[a:b, h] @ k[h // group].T * scale, -np.inf)
            p = np.exp(s - s.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out[a:b, h] = p @ v[h // group]
            weight[a:b, h] = p @ np.abs(v[h // group])
    return out, weight


def prepare_step(context_lens, query_lens, block_table, free_blocks, num_free: int,
                 block_size: int, max_tokens: int):
    """One step's metadata, request by request and token by token: (block_table, seq_lens,
    cu_seqlens_q, slot_mapping, positions, num_free)."""
    table = np.array(block_table, np.int64)
    free = [int(x) for x in np.asarray(free_blocks)[:num_free]]
    seq_lens, cu = [], [0]
    slots, positions = [], []
    for i, (c, q) in enumerate(zip(context_lens, query_lens)):
        held = -(-int(c) // block_size)
        room = held * block_size
        for p in range(int(c), int(c) + int(q)):
            if p // block_size >= held:
                table[i, p // block_size] = free.pop() if free else -1
                held += 1
                if table[i, p // block_size] >= 0:
                    room = held * block_size
            blk = table[i, p // block_size]
            slots.append(int(blk) * block_size + p % block_size if blk >= 0 else -1)
            positions.append(p)
        seq_lens.append(min(int(c) + int(q), room))
        cu.append(cu[-1] + int(q))
    pad = max_tokens - len(slots)
    i32 = lambda a: np.array(a, np.int32)  # noqa: E731
    return (i32(table), i32(seq_lens), i32(cu), i32(slots + [-1] * pad),
            i32(positions + [0] * pad), len(free))


def release_blocks(finished, seq_lens, block_table, free_blocks, num_free: int, block_size: int):
    """(free_blocks, seq_lens, num_free) after the finished rows gave their blocks back."""
    free = np.array(free_blocks)
    lens = np.array(seq_lens)
    for i in np.nonzero(np.asarray(finished))[0]:
        for j in range(-(-int(lens[i]) // block_size)):
            free[num_free] = block_table[i, j]
            num_free += 1
        lens[i] = 0
    return free, lens, num_free
