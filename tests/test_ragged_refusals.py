"""Refusals of the ragged serving path's entry points: arguments are checked before any launch. No GPU needed."""
import ctypes

import numpy as np
import pytest
import torch

import bit_kv_cache_seeded_b200 as kvq
from bit_kv_cache_seeded_b200 import build

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    build.build()
    return kvq.load()


def ptr(i, off=0):
    return ctypes.c_void_p(0x10000 * (i + 1) + off)


def refused(lib, call, args, status):
    n = kvq.kvq_kernel_launches()
    assert call(*args) == status
    assert kvq.kvq_kernel_launches() == n


def test_extend_block_table_arguments(lib):
    #        held    new     batch free    n   cursor table   pps start   ctx     taken   stream
    good = [ptr(0), ptr(1), 2, ptr(2), 10, ptr(3), ptr(4), 8, ptr(5), ptr(6), ptr(7), None]

    def bad(i, value, status=INVALID):
        refused(lib, lib.kvq_extend_block_table, good[:i] + [value] + good[i + 1:], status)
    for i in (0, 1, 3, 6, 8, 9, 10):
        bad(i, None)                              # null
    for i in (0, 1, 3, 5, 6, 8, 9, 10):
        bad(i, ptr(i, 2), ALIGNMENT)
    bad(2, 0)
    bad(4, -1)
    bad(7, 0)
    bad(7, (1 << 24) + 1)                         # over 2^30 tokens of a sequence
    for i in (6, 8, 9, 10):
        bad(i, ptr(0))                            # an output that is an input
    bad(8, ptr(6))                                # two outputs in one place


def test_slot_map_arguments(lib):
    #        held    start   ctx   batch table pps n_pages n_tokens ids  pos     slots   stream
    good = [ptr(0), ptr(1), ptr(2), 2, ptr(3), 8, 10, 5, ptr(4), ptr(5), ptr(6), None]

    def bad(i, value, status=INVALID):
        refused(lib, lib.kvq_slot_map, good[:i] + [value] + good[i + 1:], status)
    for i in (0, 1, 2, 4, 10):
        bad(i, None)
    for i in (0, 1, 2, 4, 8, 9):
        bad(i, ptr(i, 2), ALIGNMENT)
    bad(10, ptr(10, 4), ALIGNMENT)
    for i, v in ((3, 0), (5, 0), (6, 0), (7, -1)):
        bad(i, v)
    for i in (8, 9, 10):
        bad(i, ptr(1))
    bad(8, ptr(5))
    refused(lib, lib.kvq_slot_map, [None, None, None, 2, None, 8, 10, 0, None, None, None, None], OK)  # no tokens


def test_cache_calls_without_a_cache(lib):
    one = ctypes.c_size_t()
    refused(lib, lib.kvq_quantize_slots, [None, ptr(0), ptr(1), 0, ptr(2), 1, None], INVALID)
    refused(lib, lib.kvq_cache_set_lengths, [None, ptr(0), None], INVALID)
    refused(lib, lib.kvq_chunk_workspace_bytes, [None, 0, 1, ctypes.byref(one)], INVALID)
    refused(lib, lib.kvq_chunk_attention, [None, ptr(0), 0, 1, ptr(1), None, ptr(2), ptr(3), 1 << 20, None], INVALID)


def test_host_tensors_are_refused(lib):
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        kvq.kvq_extend_block_table(i32(2), i32(2), i32(4), i32(4).view(2, 2), i32(3), i32(2), i32(2))
    with pytest.raises(ValueError):
        kvq.kvq_slot_map(i32(2), i32(3), i32(2), i32(4).view(2, 2), 4, None, None, torch.zeros(3, dtype=torch.int64))
    x = torch.zeros(3, 2, 128)
    with pytest.raises(ValueError):
        kvq.kvq_quantize_slots(None, x, x, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        kvq.kvq_chunk_attention(None, x, i32(2), None, x, x)


def test_cache_object_checks_shapes(lib):
    """KvqCache's methods refuse tensors that do not fit the configuration, which the library cannot see."""
    c = object.__new__(kvq.KvqCache)
    c.batch, c.cfg, c.handle = 3, kvq.make_cfg(n_q_heads=8, n_kv_heads=2), None
    x, slots = torch.zeros(5, 2, 128), torch.zeros(5, dtype=torch.int64)
    start = torch.zeros(4, dtype=torch.int32)
    for K, V in ((x[:, :1], x[:, :1]), (x, x[:4]), (x[..., :64], x[..., :64]), (x[0], x[0])):
        with pytest.raises(ValueError):
            c.quantize_slots(K, V, slots)
    q = torch.zeros(5, 8, 128)
    for args in ((q[:, :4], start), (q[0], start), (q, start[:3]), (q, start, start[:2])):
        with pytest.raises(ValueError):
            c.chunk_attention(*args)
    with pytest.raises(TypeError):
        c.chunk_attention(q.half(), start)
    for lens in ([1, 2], [[1, 2, 3]], [1.5, 2, 3], [1, 2, 2 ** 31], np.zeros(4, dtype=int)):
        with pytest.raises(ValueError):
            c.set_lengths(lens)
