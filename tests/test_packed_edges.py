"""CPU checks of packed attention's size functions at what its calls refuse."""
import pytest

import paged_kv_attention_03_gb300 as pa

FAKE = 0x10000


def _backward(total_q, total_k, num_seqs, heads, buckets, distance):
    lib = pa.load()
    return lib.pa_varlen_attn_backward(FAKE, FAKE, FAKE, FAKE if buckets else None, heads * 64, heads * 64, heads * 64, FAKE, FAKE, FAKE, FAKE,
                                       FAKE, FAKE, heads * 64, heads * 64, heads * 64, FAKE, FAKE, num_seqs, total_q, total_k, 128, 128, heads,
                                       heads, 64, 0, 0.125, FAKE if buckets else None, buckets, distance, None, 0, None)


@pytest.mark.parametrize("sizes", [
    (100, 90, 3, 8, 32, 16), (100, 90, 3, 8, 1, 10), (100, 90, 3, 8, 129, 4000), (100, 90, 3, 8, 32, 32769), (1 << 30, 90, 3, 8, 0, 0),
    (100, 1 << 30, 3, 8, 0, 0), (100, 90, 65536, 8, 0, 0), (100, 90, -1, 8, 0, 0), (100, 90, 3, 0, 0, 0), (100, -1, 3, 8, 0, 0),
    (100, 90, 3, 8, -1, 0), ((1 << 30) - 1, 90, 3, 512, 0, 0)])
def test_backward_size_of_what_the_call_refuses(sizes):
    assert pa.pa_varlen_attn_backward_workspace_size(*sizes) == 0
    assert _backward(*sizes) != pa.PA_OK


@pytest.mark.parametrize("sizes", [(100, 90, 3, 8, 0, 0), (100, 90, 3, 8, 32, 128), (1, 0, 1, 1, 2, 2), (0, 5, 65535, 1, 0, 0)])
def test_backward_size_of_what_it_takes(sizes):
    assert pa.pa_varlen_attn_backward_workspace_size(*sizes) >= pa.pa_relative_bias_workspace_size(*sizes[3:])
    assert pa.pa_varlen_attn_backward_workspace_size(*sizes) > 0
