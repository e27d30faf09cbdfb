"""What is measured of attention with a learned relative position bias, and the plain form of each operator.

The operators:

* ``attend``: attention of packed sequences of different lengths on plain K/V, causal, grouped heads, with the logarithm
  of the softmax denominators (``pa_varlen_attn``);
* ``train``: the same and its gradient, as a training step runs them (``pa_varlen_attn``, ``pa_varlen_attn_backward``);
* ``prefill``: packed prompts over the paged cache, with the bias (``pa_varlen_prefill_bias``);
* ``decode``: one query per sequence over the paged cache, with the bias (``pa_decode_bias``).

The bias: a table ``[num_buckets, num_heads]``; a query at position p adds entry ``[bucket(p - j), head]`` to the logit of
key j.  With m = num_buckets // 2, distances below m have a bucket each, and a distance n beyond has bucket
m + floor(ln(n / m) / ln(max_distance / m) * (num_buckets - m)), at most num_buckets - 1.
"""
import torch

own = False


# ------------------------------------------------------------------ cases ---
def listed():
    return [
        # Scoring three short texts, 8/2 heads of 64, no bias: latency.
        {"name": "attend short", "op": "attend", "prompts": 3, "low": 5, "high": 60, "ctx_low": 0, "ctx_high": 0, "heads": 8,
         "kv_heads": 2, "dim": 64, "window": 0, "buckets": 0, "distance": 0},
        # The varlen prefill workload's prompts, scored without a cache: 16 of 128 to 2048 tokens.
        {"name": "attend varlen", "op": "attend", "prompts": 16, "low": 128, "high": 2048, "ctx_low": 0, "ctx_high": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "window": 0, "buckets": 32, "distance": 128},
        # A training step on two short sequences: latency.
        {"name": "train tiny", "op": "train", "prompts": 2, "low": 33, "high": 100, "ctx_low": 0, "ctx_high": 0, "heads": 8,
         "kv_heads": 2, "dim": 64, "window": 0, "buckets": 32, "distance": 128},
        # Many short sequences packed, every head with its own keys, heads of 64.
        {"name": "train sentences", "op": "train", "prompts": 64, "low": 17, "high": 512, "ctx_low": 0, "ctx_high": 0, "heads": 12,
         "kv_heads": 12, "dim": 64, "window": 0, "buckets": 32, "distance": 128},
        # Packed documents of 128 to 2048 tokens, 32/8 heads of 128.
        {"name": "train varlen", "op": "train", "prompts": 16, "low": 128, "high": 2048, "ctx_low": 0, "ctx_high": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "window": 0, "buckets": 32, "distance": 128},
        # Two long documents, no bias.
        {"name": "train long", "op": "train", "prompts": 2, "low": 6000, "high": 8192, "ctx_low": 0, "ctx_high": 0, "heads": 32,
         "kv_heads": 8, "dim": 128, "window": 0, "buckets": 0, "distance": 0},
        # The smallest decode: four short sequences, 8/2 heads of 64 (latency).
        {"name": "decode tiny", "op": "decode", "batch": 4, "heads": 8, "kv_heads": 2, "dim": 64, "block": 16, "low": 17,
         "high": 100, "window": 0, "buckets": 32, "distance": 128},
        # The batched decode workload: 64 requests of 512 to 4096 keys, 32/8 heads.
        {"name": "decode batched", "op": "decode", "batch": 64, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16,
         "low": 512, "high": 4096, "window": 0, "buckets": 32, "distance": 128},
        # The long decode workload: 8 requests of 32k to 131k keys, 40/8 heads.
        {"name": "decode long", "op": "decode", "batch": 8, "heads": 40, "kv_heads": 8, "dim": 128, "block": 16,
         "low": 32768, "high": 131072, "window": 0, "buckets": 64, "distance": 2048},
        # A few short prompts with a cached context, odd lengths, pages of 64.
        {"name": "prefill few chunks", "op": "prefill", "prompts": 3, "low": 37, "high": 301, "ctx_low": 0, "ctx_high": 700,
         "decodes": 0, "heads": 32, "kv_heads": 8, "dim": 128, "block": 64, "window": 0, "buckets": 32, "distance": 128},
        # The varlen prefill workload: 16 prompts of 128 to 2048 tokens.
        {"name": "prefill varlen", "op": "prefill", "prompts": 16, "low": 128, "high": 2048, "ctx_low": 0, "ctx_high": 0,
         "decodes": 0, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "window": 0, "buckets": 32, "distance": 128},
        # Chunked prefill beside decodes in one call, with a sliding window and buckets over a longer distance.
        {"name": "prefill mixed window", "op": "prefill", "prompts": 4, "low": 512, "high": 512, "ctx_low": 1024,
         "ctx_high": 4096, "decodes": 24, "heads": 32, "kv_heads": 8, "dim": 128, "block": 16, "window": 2048, "buckets": 64,
         "distance": 1024},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return int(round(float(low) * (float(high) / low) ** rng.random()))


def draw(rng):
    op = rng.choice(("attend", "train", "train", "train", "decode", "decode", "prefill"))
    dim = rng.choice((64, 128, 128))
    kv_heads = rng.choice((1, 2, 4, 8))
    group = rng.choice((1, 2, 4, 5, 7, 8, 16))
    group = min(group, 40 // kv_heads)
    case = {"op": op, "heads": kv_heads * group, "kv_heads": kv_heads, "dim": dim}
    buckets = rng.choice((8, 16, 32, 32, 64, 2 * rng.randint(2, 50)))
    distance = rng.choice((128, 128, _spread(rng, buckets // 2 + 1, 4000)))
    case |= {"buckets": buckets, "distance": max(distance, buckets // 2 + 1)}
    if op == "decode":
        high = _spread(rng, 30, 60000)
        batch = _spread(rng, 1, max(2, min(700, 8 * 131072 * 8 // (2 * high * kv_heads))))
        return case | {"batch": batch, "block": rng.choice((16, 32, 64)), "low": 1 + high // rng.randint(2, 20), "high": high,
                       "window": rng.choice((0, 0, 1 + rng.randint(1, high)))}
    high = _spread(rng, 3, 3000)
    ctx = rng.choice((0, _spread(rng, 1, 2000)))
    prompts = _spread(rng, 1, max(2, min(100, int(16 * 32 * 2048 * 2048 // (2 * case["heads"] * high * (high + ctx))))))
    case |= {"prompts": prompts, "low": 1 + high // rng.randint(2, 9), "high": high, "ctx_low": ctx // 2, "ctx_high": ctx,
             "window": rng.choice((0, 0, 1 + rng.randint(1, high + ctx)))}
    if op == "prefill":
        return case | {"decodes": rng.choice((0, rng.randint(1, 9))), "block": rng.choice((16, 32, 64))}
    if rng.random() < 0.25:
        case |= {"buckets": 0, "distance": 0}
    return case


# ---------------------------------------------------------------- inputs ---
def _between(low, high, n, g):
    """n whole numbers between low and high: the same ones for every seed, so that outputs keep their shapes, in the seed's order."""
    n_ = torch.randint(low, high + 1, (n,), generator=torch.Generator().manual_seed(n), dtype=torch.int64)
    return n_[torch.randperm(n, generator=g)]


def _lengths(case, g):
    """(new tokens, keys) of each sequence; the decodes of a prefill case stand behind its prompts."""
    if case["op"] == "decode":
        keys = _between(case["low"], case["high"], case["batch"], g)
        return torch.ones_like(keys), keys
    decodes = case.get("decodes", 0)
    new = torch.cat([_between(case["low"], case["high"], case["prompts"], g), torch.ones(decodes, dtype=torch.int64)])
    return new, new + _between(case["ctx_low"], case["ctx_high"], case["prompts"] + decodes, g)


def _offsets(n):
    return torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    d = torch.Generator(device="cuda").manual_seed(seed + 1)
    dev = lambda t: t.to(torch.int32).cuda()  # noqa: E731
    normal = lambda *shape: torch.randn(*shape, generator=d, device="cuda").bfloat16()  # noqa: E731
    heads, hkv, dim = case["heads"], case["kv_heads"], case["dim"]
    new, keys = _lengths(case, g)
    cu_q, cu_k = _offsets(new), _offsets(keys)
    s = {"case": case, "new": new.tolist(), "keys": keys.tolist(), "cu_seqlens_q": dev(cu_q), "max_q": int(new.max()),
         "max_k": int(keys.max()), "scale": dim ** -0.5, "q": normal(int(cu_q[-1]), heads, dim)}
    if case["buckets"]:
        s["bias"] = torch.randn(case["buckets"], heads, generator=d, device="cuda")
    if case["op"] in ("attend", "train"):
        s |= {"cu_seqlens_k": dev(cu_k), "k": normal(int(cu_k[-1]), hkv, dim), "v": normal(int(cu_k[-1]), hkv, dim)}
        if case["op"] == "train":
            s["dout"] = normal(int(cu_q[-1]), heads, dim)
        return s
    bs = case["block"]
    blocks = (keys + bs - 1) // bs
    num_blocks = int(blocks.sum()) + 9
    perm = torch.randperm(num_blocks, generator=g, dtype=torch.int64)
    col = torch.arange(int(blocks.max()))
    at = ((blocks.cumsum(0) - blocks)[:, None] + col).clamp(max=num_blocks - 1)
    s |= {"seq_lens": dev(keys), "block_table": dev(torch.where(col < blocks[:, None], perm[at], -1)),
          "k_cache": torch.empty(num_blocks, bs, hkv, dim, dtype=torch.bfloat16, device="cuda"),
          "v_cache": torch.empty(num_blocks, bs, hkv, dim, dtype=torch.bfloat16, device="cuda")}
    slab = max(1, (1 << 28) // (hkv * bs * dim))
    for cache in (s["k_cache"], s["v_cache"]):
        for b in range(0, num_blocks, slab):
            cache[b:b + slab] = torch.randn(cache[b:b + slab].shape, generator=d, device="cuda")
    return s


# ------------------------------------------------------------ plain forms ---
def _buckets(n, buckets, distance):
    """The bucket of each distance; borders in 64 bits, a distance on a border counted as beyond it."""
    m = buckets // 2
    step = torch.arange(1, buckets - m, dtype=torch.float64, device=n.device) / (buckets - m)
    border = m * (float(distance) / m) ** step * (1 - 1e-12)
    return torch.where(n < m, n, m + (n[..., None] >= border).sum(-1)).clamp(min=0)


def _by_bucket(case, count, device):
    return _buckets(torch.arange(count, device=device), case["buckets"], case["distance"])


def _mask(case, new, keys, device):
    """What the last `new` positions of a sequence of `keys` see, and the distances."""
    far = (keys - new + torch.arange(new, device=device))[:, None] - torch.arange(keys, device=device)
    see = far >= 0
    if case["window"] > 0:
        see = see & (far < case["window"])
    return see, far


def _plain_sequence(s, q, k, v, dout, dbias):
    """One sequence: q [new, heads, dim], k / v [keys, kv heads, dim] -> out, lse (and dq, dk, dv; dbias is added to)."""
    case = s["case"]
    new, heads, dim = q.shape
    keys, hkv, _ = k.shape
    group = heads // hkv
    see, far = _mask(case, new, keys, q.device)
    by = _by_bucket(case, max(keys, 1), q.device) if case["buckets"] else None
    parts = []
    step = max(1, (1 << 28) // (group * new * keys))  # kv heads at a time
    for h in range(0, hkv, step):
        kh = k[:, h:h + step].float().transpose(0, 1)[:, None]
        vh = v[:, h:h + step].float().transpose(0, 1)[:, None]
        n = kh.shape[0]
        split = lambda x: x[:, h * group:(h + n) * group].float().transpose(0, 1).unflatten(0, (n, group))  # noqa: E731
        qh = split(q)
        p = (qh @ kh.transpose(2, 3)) * s["scale"]
        if by is not None:
            table = s["bias"][by][:, h * group:(h + n) * group].T.unflatten(0, (n, group))  # [n, group, keys] by distance
            p = p + table[..., far.clamp(min=0)]
        p = p.masked_fill(~see, float("-inf"))
        top = p.amax(-1, keepdim=True).clamp(min=-3e38)
        p = torch.exp(p - top)
        total = p.sum(-1, keepdim=True)
        lse = (top + torch.log(total)).squeeze(-1)
        p = p / total.clamp(min=1e-30)
        o = p @ vh
        back = lambda x: x.flatten(0, 1).transpose(0, 1)  # noqa: E731
        if dout is None:
            parts.append((back(o), lse.flatten(0, 1).T))
            continue
        do = split(dout)
        dv = (p.transpose(2, 3) @ do).sum(1)
        ds = p * (do @ vh.transpose(2, 3) - (do * o).sum(-1, keepdim=True))
        dq = ds @ kh * s["scale"]
        dk = (ds.transpose(2, 3) @ qh).sum(1) * s["scale"]
        parts.append((back(o), lse.flatten(0, 1).T, back(dq), dk.transpose(0, 1), dv.transpose(0, 1)))
        if by is not None:
            # Sums over each diagonal: row r is shifted by r, then columns are summed; buckets in 64 bits.
            ds = torch.nn.functional.pad(ds.flatten(0, 1).flip(-1), (0, new))
            ds = ds.flatten(1)[:, : new * (new + keys - 1)].unflatten(1, (new, new + keys - 1))
            diagonal = ds.sum(1, dtype=torch.float64)[:, new - 1:]
            hit = (by[:, None] == torch.arange(case["buckets"], device=q.device)).double()
            dbias[:, h * group:(h + n) * group] += (diagonal @ hit[: diagonal.shape[1]]).T
    return [torch.cat(x, dim=1) for x in zip(*parts)]


def _plain_packed(s):
    train = s["case"]["op"] == "train"
    dbias = torch.zeros(s["bias"].shape, dtype=torch.float64, device="cuda") if train and "bias" in s else None
    parts, a, b = [], 0, 0
    for new, keys in zip(s["new"], s["keys"]):
        parts.append(_plain_sequence(s, s["q"][a:a + new], s["k"][b:b + keys], s["v"][b:b + keys],
                                     s["dout"][a:a + new] if train else None, dbias))
        a, b = a + new, b + keys
    got = [torch.cat(x) for x in zip(*parts)]
    r = {"out": got[0].bfloat16(), "lse": got[1]}
    if train:
        r |= {"dq": got[2].bfloat16(), "dk": got[3].bfloat16(), "dv": got[4].bfloat16()}
        if dbias is not None:
            r["dbias"] = dbias.float()
    return r


def _plain_paged(s):
    parts, a, bs = [], 0, s["case"]["block"]
    for i, (new, keys) in enumerate(zip(s["new"], s["keys"])):
        blocks = s["block_table"][i, : (keys + bs - 1) // bs].long()
        k, v = (c[blocks].flatten(0, 1)[:keys] for c in (s["k_cache"], s["v_cache"]))
        parts.append(_plain_sequence(s, s["q"][a:a + new], k, v, None, None)[0])
        a += new
    return torch.cat(parts).bfloat16()


def _own(s):
    import paged_kv_attention_03_gb300 as pa
    case = s["case"]
    bias, distance, w = s.get("bias"), case["distance"], case["window"]
    if case["op"] == "decode":
        return pa.pa_decode_bias(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["max_k"], s["scale"],
                                 bias, distance, w)
    if case["op"] == "prefill":
        return pa.pa_varlen_prefill_bias(s["q"], s["k_cache"], s["v_cache"], s["cu_seqlens_q"], s["seq_lens"], s["block_table"],
                                         s["max_q"], s["max_k"], s["scale"], bias, distance, w)
    out, lse = pa.pa_varlen_attn(s["q"], s["k"], s["v"], s["cu_seqlens_q"], s["cu_seqlens_k"], s["max_q"], s["max_k"], s["scale"],
                                 w, bias=bias, max_distance=distance)
    r = {"out": out, "lse": lse}
    if case["op"] == "train":
        r["dq"], r["dk"], r["dv"], dbias = pa.pa_varlen_attn_backward(
            s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu_seqlens_q"], s["cu_seqlens_k"], s["max_q"], s["max_k"], s["scale"],
            w, bias=bias, max_distance=distance)
        if bias is not None:
            r["dbias"] = dbias
    return r


def run(s):
    if own:
        return _own(s)
    return _plain_packed(s) if s["case"]["op"] in ("attend", "train") else _plain_paged(s)


# ------------------------------------------------------------------ work ---
def work(case):
    """Bytes and operations of one pass: 4 dim operations a visible pair and head forward (two products), 10 dim more backward (five)."""
    new, keys = (n.double() for n in _lengths(case, torch.Generator().manual_seed(0)))
    heads, hkv, dim = case["heads"], case["kv_heads"], case["dim"]
    w = torch.full_like(keys, case["window"] if case["window"] > 0 else 1e18)
    ctx = keys - new
    # Row r sees min(ctx + r + 1, w) keys: r + 1 of them grow until the window is full.
    grow = (w - ctx).clamp(min=0).minimum(new)
    pairs = float((grow * ctx + grow * (grow + 1) / 2 + (new - grow) * w.minimum(keys)).sum())
    read = float(torch.minimum(keys, new + w - 1).sum())
    tokens = float(new.sum())
    q_bytes, kv_bytes = 2 * tokens * heads * dim, 4 * read * hkv * dim
    bias = 4 * case["buckets"] * heads
    flops = 4 * heads * dim * pairs
    if case["op"] in ("decode", "prefill"):
        return {"bytes": 2 * q_bytes + kv_bytes + bias, "flops": flops}
    lse = 4 * tokens * heads
    if case["op"] == "attend":
        return {"bytes": 2 * q_bytes + kv_bytes + lse + bias, "flops": flops}
    # a step: q, k, v, dout and the bias read; out, lse and the gradients written
    return {"bytes": 4 * q_bytes + 2 * kv_bytes + lse + 2 * bias, "flops": flops * 3.5}


# ------------------------------------------------------------- 64 bits ---
def _first_distances(buckets, distance):
    """The smallest distance of each bucket, by whole numbers: n >= m (distance / m)^(j / r) is n^r >= m^(r - j) distance^j."""
    m = buckets // 2
    r = buckets - m
    first = list(range(m))
    for j in range(r):
        want = m ** (r - j) * distance ** j
        low, high = m, distance
        while low < high:
            mid = (low + high) // 2
            low, high = (low, mid) if mid ** r >= want else (mid + 1, high)
        first.append(low)
    return first


def exact(case, seed):
    s = prepare(case, seed)
    new, keys = s["new"], s["keys"]
    heads, hkv, dim, w = case["heads"], case["kv_heads"], case["dim"], case["window"]
    train, packed = case["op"] == "train", case["op"] in ("attend", "train")
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out, lse = zeros(s["q"].shape), zeros(s["q"].shape[:2])
    if train:
        dq, dk, dv = zeros(s["q"].shape), zeros(s["k"].shape), zeros(s["k"].shape)
        dbias = zeros(case["buckets"], heads)
    if case["buckets"]:
        first = torch.tensor(_first_distances(case["buckets"], case["distance"]), device="cuda")
    a = b = 0
    for i, (t, n) in enumerate(zip(new, keys)):
        if packed:
            k, v = s["k"][b:b + n], s["v"][b:b + n]
        else:
            slot = torch.arange(n, device="cuda")
            block = s["block_table"][i].long()[slot // case["block"]]
            k, v = s["k_cache"][block, slot % case["block"]], s["v_cache"][block, slot % case["block"]]
        pos = torch.arange(n - t, n, device="cuda")[:, None]
        key = torch.arange(n, device="cuda")[None]
        hidden = key > pos
        if w > 0:
            hidden = hidden | (key <= pos - w)
        if case["buckets"]:
            bucket = torch.searchsorted(first, (pos - key).clamp(min=0), right=True) - 1
        for h in range(heads):
            qh, kh, vh = s["q"][a:a + t, h].double(), k[:, h * hkv // heads].double(), v[:, h * hkv // heads].double()
            logit = s["scale"] * (qh @ kh.T)
            if case["buckets"]:
                logit += s["bias"][:, h].double()[bucket]
            logit[hidden] = float("-inf")
            lse[a:a + t, h] = torch.logsumexp(logit, dim=1)
            p = torch.softmax(logit, dim=1)
            out[a:a + t, h] = p @ vh
            if not train:
                continue
            do = s["dout"][a:a + t, h].double()
            dp = do @ vh.T
            ds = p * (dp - (p * dp).sum(dim=1, keepdim=True))
            dq[a:a + t, h] = s["scale"] * (ds @ kh)
            dk[b:b + n, h * hkv // heads] += s["scale"] * (ds.T @ qh)
            dv[b:b + n, h * hkv // heads] += p.T @ do
            if case["buckets"]:
                ds[hidden] = 0.0
                # key by key, from the far end of each row: rows of equal distance lie on a diagonal
                flat = torch.zeros(n, dtype=torch.float64, device="cuda")
                for r in range(0, t, 1024):
                    part = ds[r:r + 1024]
                    width = n + part.shape[0]
                    skew = zeros(part.shape[0], width)
                    skew[:, : n] = part.flip(1)
                    skew = skew.flatten()[: part.shape[0] * (width - 1)].view(part.shape[0], width - 1).sum(0)
                    d0 = n - t + r - (n - 1)  # distance of column 0
                    lo, hi = max(0, -d0), min(width - 1, n - d0)
                    flat[d0 + lo:d0 + hi] += skew[lo:hi]
                dbias[:, h].index_add_(0, torch.searchsorted(first, torch.arange(n, device="cuda"), right=True) - 1, flat)
        a, b = a + t, b + n
    if not packed:
        return out
    r = {"out": out, "lse": lse}
    if train:
        r |= {"dq": dq, "dk": dk, "dv": dv}
        if case["buckets"]:
            r["dbias"] = dbias
    return r
