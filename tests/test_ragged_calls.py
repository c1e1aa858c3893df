"""The ragged serving path's calls as far as they need no GPU: refusals, and what the Python side hands to the library."""
import ctypes

import pytest
import torch

import bit_kv_cache_seeded_b200 as kvq
from bit_kv_cache_seeded_b200 import build

INVALID = 1


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kvq.load()


def ptr(i):
    return ctypes.c_void_p(0x10000 * (i + 1))


def bare_cache(batch=3, n_q_heads=8, n_kv_heads=2):
    c = object.__new__(kvq.KvqCache)
    c.batch, c.cfg, c.handle = batch, kvq.make_cfg(n_q_heads=n_q_heads, n_kv_heads=n_kv_heads), None
    return c


def test_append_of_request_rows_refuses(lib):
    n = kvq.kvq_kernel_launches()
    assert lib.kvq_quantize_slots_rows(None, ptr(0), ptr(1), 0, ptr(2), 1, ptr(3), None) == INVALID
    assert lib.kvq_quantize_slots_rows(ptr(9), ptr(0), ptr(1), 0, ptr(2), 1, None, None) == INVALID
    x, slots = torch.zeros(5, 2, 128), torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="seq_start"):
        bare_cache().quantize_slots(x, x, slots, seq_start=torch.zeros(3, dtype=torch.int32))
    assert kvq.kvq_kernel_launches() == n


def test_attention_with_lengths_before_the_step_refuses(lib):
    n = kvq.kvq_kernel_launches()
    args = [None, ptr(0), 0, 1, ptr(1), None, ptr(2), ptr(3), ptr(4), 1 << 20, None]
    assert lib.kvq_chunk_attention_held(*args) == INVALID
    assert lib.kvq_chunk_attention_held(ptr(9), *args[1:6], None, *args[7:]) == INVALID
    with pytest.raises(ValueError, match="held"):
        bare_cache().chunk_attention(torch.zeros(5, 8, 128), torch.zeros(4, dtype=torch.int32),
                                     held=torch.zeros(4, dtype=torch.int32))
    assert kvq.kvq_kernel_launches() == n
