"""CPU checks behind the GPU tests of split key tiles: that their cases have what they are for, and that the 64-bit values they
are compared with are the oracle's."""
import numpy as np
import pytest
import torch

from _packed import SPLIT, constant, key_items, parts_before_another_head, values
from oracle import relative


def test_the_model_counts_for_this_gpu():
    assert constant("kPlanSms", "pa_internal.h") == 152


@pytest.mark.parametrize("name", SPLIT)
def test_cases_have_parts_before_another_head(name):
    sq, sk, heads, hkv, _, window, _, _ = SPLIT[name]
    blocks = key_items(sq, sk, heads, hkv, window)
    assert hkv > 1 and sum(map(len, blocks)) > len(blocks) == 152
    assert parts_before_another_head(sq, sk, heads, hkv, window) > 0


def test_parts_cover_every_tile_and_head_once():
    sq, sk, heads, hkv, _, window, _, _ = SPLIT["three"]
    items = [x for b in key_items(sq, sk, heads, hkv, window) for x in b]
    assert len(set(items)) == len(items)
    tiles = sum(-(-n // 128) for n in sk)
    for tile in range(tiles):
        for h in range(hkv):
            parts = [x for x in items if x[0] == tile and x[3] == h]
            assert sorted(p for _, p, _, _ in parts) == list(range(parts[0][2]))


@pytest.mark.parametrize("window,buckets,distance", [(0, 0, 0), (0, 6, 9), (5, 8, 12)])
def test_values_are_the_oracles(window, buckets, distance):
    g = torch.Generator().manual_seed(window + buckets)
    normal = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    cu_q, cu_k = np.array([0, 20, 20, 33, 37]), np.array([0, 27, 33, 42, 42])  # more keys, no queries, more queries, no keys
    q, k, v, dout = normal(37, 4, 8), normal(42, 2, 8), normal(42, 2, 8), normal(37, 4, 8)
    bias = normal(buckets, 4) if buckets else None
    if buckets:
        bias[0, 1] = float("-inf")
    got = values(q, k, v, cu_q, cu_k, window, 0.6, bias, distance, dout)
    want = relative.attention(q.numpy(), k.numpy(), v.numpy(), cu_q, cu_k, window, 0.6, None if bias is None else bias.numpy(), distance,
                              dout.numpy())
    for name, x in want.items():
        if name == "logit" or (name.startswith("dv_") and name != "dv_abs"):  # (the oracle's logit has |s| in place of |bias|)
            continue
        # sums of at most 100 terms of order 10: 1e-13; an error term of a key that a row does not see may be left out
        np.testing.assert_allclose(got[name].numpy(), x, rtol=1e-12, atol=1e-12, err_msg=name)
    assert (got["ds_abs"] >= 0).all() and (got["ds_abs"] > 0).any()
