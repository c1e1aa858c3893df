"""The ragged serving path's calls as far as they need no GPU: refusals, and what the Python side hands to the library."""
import contextlib
import ctypes

import threading
import time

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
    c.chunk_workspaces, c.chunk_lock = {}, threading.Lock()
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


class Streams:
    """Stands in for torch's streams: knows the current one, and on which every tensor was made."""

    def __init__(self, monkeypatch):
        self.current, self.made, self.calls = "current", [], []
        for name in ("empty", "empty_like"):
            monkeypatch.setattr(torch, name, self._recorded(getattr(torch, name)))
        monkeypatch.setattr(torch.cuda, "stream", self._switched)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(kvq, "_stream", lambda s=None: s or self.current)
        monkeypatch.setattr(kvq, "_here", lambda *args, **tensors: None)

    def _recorded(self, make):
        def made(*args, **kw):
            t = make(*args, **kw)
            self.made.append((t, self.current))
            return t
        return made

    @contextlib.contextmanager
    def _switched(self, stream):
        before, self.current = self.current, stream
        yield
        self.current = before

    def of(self, tensor):
        return next(s for t, s in self.made if t is tensor)


def test_attention_on_a_named_stream_makes_its_tensors_there(lib, monkeypatch):
    """Memory of another stream may be in use by work that the named one does not wait for."""
    streams, seen = Streams(monkeypatch), []
    monkeypatch.setattr(kvq, "kvq_chunk_workspace_bytes", lambda handle, dtype, n: 64)
    monkeypatch.setattr(kvq, "kvq_chunk_attention", lambda h, q, start, ctx, out, ws, stream, held=None: seen.append((out, ws, stream)))
    c, q, start = bare_cache(), torch.zeros(5, 8, 128), torch.zeros(4, dtype=torch.int32)
    for stream in ("side", None):
        out = c.chunk_attention(q, start, stream=stream)
        used, ws, at = seen[-1]
        assert used is out and at == stream and streams.current == "current"
        assert streams.of(out) == streams.of(ws) == (stream or "current")
    mine = torch.zeros_like(q)
    assert c.chunk_attention(q, start, out=mine, stream="side") is mine


def test_decode_calls_on_a_named_stream_make_their_tensors_there(lib, monkeypatch):
    streams, seen = Streams(monkeypatch), []
    for name in ("kvq_decode_attention", "kvq_decode_step", "kvq_decode_partials", "kvq_decode_step_host"):
        monkeypatch.setattr(kvq, name, lambda *args, name=name: seen.append((name, args)))
    monkeypatch.setattr(kvq, "kvq_partial_floats", lambda handle: 130)
    monkeypatch.setattr(kvq, "kvq_step_staging_bytes", lambda handle, dtype: 64)
    monkeypatch.setattr(torch.Tensor, "pin_memory", lambda t: t)
    c, q, kv = bare_cache(), torch.zeros(3, 8, 128), torch.zeros(3, 2, 1, 128)
    c.out_dim, c.workspace = 128, torch.zeros(64, dtype=torch.uint8)
    for stream in ("side", None):
        c.staging = None
        made = [c.decode(q, stream=stream), c.step(kv, kv, q, stream=stream), c.decode_partials(q, stream=stream)]
        c.step_host(kv, kv, q, stream=stream)
        assert [streams.of(t) for t in (*made, c.staging)] == [stream or "current"] * 4
        assert streams.current == "current"
    assert [name for name, _ in seen[:4]] == ["kvq_decode_attention", "kvq_decode_step", "kvq_decode_partials", "kvq_decode_step_host"]


def test_context_parallel_decode_on_a_named_stream_exchanges_there(lib, monkeypatch):
    from bit_kv_cache_seeded_b200 import context_parallel
    streams, seen = Streams(monkeypatch), []
    monkeypatch.setattr(kvq, "kvq_partial_floats", lambda handle: 130)
    monkeypatch.setattr(kvq, "kvq_decode_partials", lambda *args: seen.append(("states", args[-1])))
    monkeypatch.setattr(context_parallel, "exchange_states", lambda t, group: seen.append(("exchange", streams.current)) or t[None])
    monkeypatch.setattr(context_parallel, "kvq_combine_partials", lambda s, out, stream: seen.append(("merge", stream)))
    c, q = bare_cache(), torch.zeros(3, 8, 128)
    c.out_dim, c.workspace = 128, torch.zeros(64, dtype=torch.uint8)
    for stream in ("side", None):
        out = context_parallel.context_parallel_decode(c, q, stream=stream)
        assert streams.of(out) == (stream or "current")
    assert seen == [(n, s) for s in ("side", None) for n in ("states", "exchange", "merge")][:3] + [
        ("states", None), ("exchange", "current"), ("merge", None)]


def test_threads_that_share_a_workspace_enqueue_in_turn(lib, monkeypatch):
    """A call's kernels use its workspace one after the other: another thread's must not come between."""
    Streams(monkeypatch)
    inside, most, used = [], [], []

    def enqueue(h, q, start, ctx, out, ws, stream, held=None):
        inside.append(1)
        used.append(ws)
        time.sleep(0.02)
        most.append(len(inside))
        inside.pop()
    monkeypatch.setattr(kvq, "kvq_chunk_workspace_bytes", lambda handle, dtype, n: 64)
    monkeypatch.setattr(kvq, "kvq_chunk_attention", enqueue)
    c, q, start = bare_cache(), torch.zeros(5, 8, 128), torch.zeros(4, dtype=torch.int32)
    threads = [threading.Thread(target=lambda: [c.chunk_attention(q, start) for _ in range(3)]) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(most) == 12 and max(most) == 1
    assert all(ws is used[0] for ws in used)


def test_a_workspace_is_kept_for_its_device(lib, monkeypatch):
    """A call that is refused because its tensors are on another device than the cache leaves no workspace there for the
    next call on the same stream handle."""
    Streams(monkeypatch)
    c = bare_cache()
    wrong, right = torch.device("meta"), torch.device("cpu")
    assert c._chunk_workspace(64, wrong).device == wrong
    kept = c._chunk_workspace(64, right)
    assert kept.device == right and c._chunk_workspace(32, right) is kept


def test_attention_makes_nothing_beside_a_host_tensor(lib, monkeypatch):
    c = bare_cache()
    monkeypatch.setattr(kvq, "kvq_chunk_workspace_bytes", lambda handle, dtype, n: pytest.fail("asked for a workspace"))
    with pytest.raises(ValueError, match="CUDA tensor"):
        c.chunk_attention(torch.zeros(5, 8, 128), torch.zeros(4, dtype=torch.int32))
    assert not c.chunk_workspaces


def test_close_gives_the_workspaces_back(lib, monkeypatch):
    Streams(monkeypatch)
    monkeypatch.setattr(kvq, "kvq_cache_destroy", lambda handle: None)
    c = bare_cache()
    c.handle = 1
    c._chunk_workspace(64, torch.device("cpu"))
    assert len(c.chunk_workspaces) == 1
    c.close()
    assert c.handle is None and not c.chunk_workspaces


def test_block_tables_of_too_many_requests_are_refused(lib):
    """A block walks all requests before its own: near 2^31 of them its counter would wrap, and long before that the call
    would take minutes."""
    n = kvq.kvq_kernel_launches()
    for batch in ((1 << 20) + 1, 2 ** 31 - 8, 2 ** 31 - 1):
        assert lib.kvq_extend_block_table(ptr(0), ptr(1), batch, ptr(2), 10, None, ptr(4), 8, ptr(5), ptr(6), ptr(7), None) == INVALID
    assert kvq.kvq_kernel_launches() == n


def test_counts_of_more_than_32_bits_are_refused(lib, monkeypatch):
    """Not cut down to their low 32 bits: 2^32 + 5 new tokens are not 5."""
    monkeypatch.setattr(kvq, "_here", lambda *args, **tensors: None)
    monkeypatch.setattr(kvq, "load", lambda: pytest.fail("reached the library"))
    many = 2 ** 32 + 5
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="meta")  # noqa: E731
    x = torch.empty(many, 1, 128, device="meta")
    calls = [lambda: kvq.kvq_chunk_workspace_bytes(None, torch.float32, many),
             lambda: kvq.kvq_extend_block_table(i32(2), i32(2), i32(many), i32(2, 3), i32(3), i32(2), i32(2)),
             lambda: kvq.kvq_extend_block_table(i32(many), i32(many), i32(4), i32(many, 1), i32(many + 1), i32(many), i32(2)),
             lambda: kvq.kvq_slot_map(i32(2), i32(3), i32(2), i32(2, 3), 4, None, None, i32(many)),
             lambda: kvq.kvq_slot_map(i32(2), i32(3), i32(2), i32(2, 3), many, None, None, i32(4)),
             lambda: kvq.kvq_quantize_slots(None, x, x, i32(many)),
             lambda: kvq.kvq_chunk_attention(None, x, i32(2), None, x, i32(4))]
    for call in calls:
        with pytest.raises(ValueError, match="32 bits"):
            call()
