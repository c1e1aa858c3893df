"""Ragged serving path on the GPU: block tables and slot maps from request lengths, appends by slots, and
attention of a ragged batch of new tokens over the packed pages, each against its plain form in 64 bits."""
import numpy as np
import pytest
import torch

import bit_kv_cache_seeded_b200 as kvq
from tests._ragged import (PAGE, Batch, assert_close, causal_attention, cuda_ints, dequantised, extend_block_table, make_cfg,
                           signs_and_sketch, slot_map)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
MODES = {"2q2q": (2, True, 2, True), "3q3": (3, True, 3, False), "11": (1, False, 1, False), "2q2": (2, True, 2, False),
         "3q3q": (3, True, 3, True), "22": (2, False, 2, False), "33": (3, False, 3, False),
         # keys in token order: no tensor-core decode instance
         "1q2": (1, True, 2, False), "23q": (2, False, 3, True), "31": (3, False, 1, False)}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvq.load()


# ---- block tables and slot maps

LENGTHS = {
    "one": ([0], [1], 4, 3, None),
    "page edges": ([0, 63, 64, 65, 128, 0], [64, 1, 64, 63, 0, 0], 6, 20, 4),
    "out of pages": ([10, 64, 0, 5, 60], [200, 64, 64, 59, 500], 9, 5, None),     # later ones still need none
    "refused": ([-1, 5, 100, 2 ** 31 - 1, 7], [5, -3, 1000, 2 ** 31 - 1, 9], 8, 30, 2),
    "cursor behind": ([0, 1], [64, 1], 3, 8, 9),
    "cursor negative": ([0, 1], [64, 1], 3, 8, -1),
    "no free pages": ([0, 1], [64, 1], 3, 0, None),
}


def check_tables(held, new, pps, free, cursor):
    rng = np.random.default_rng(1)
    table = rng.integers(0, 1000, (len(held), pps)).astype(np.int32)
    dev = cuda_ints(table)
    start, ctx, taken = (cuda_ints(np.full(n, 77)) for n in (len(held) + 1, len(held), 2))
    kvq.kvq_extend_block_table(cuda_ints(held), cuda_ints(new), cuda_ints(free), dev, start, ctx, taken,
                               None if cursor is None else cuda_ints([cursor]))
    want = extend_block_table(held, new, free, cursor or 0, table)
    for got, w in zip((dev, start, ctx, taken), want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)
    n_tokens = int(min(want[1][-1], 3000)) + 7
    n_pages = 900
    outs = [cuda_ints(np.full(n_tokens, 55), t) for t in (torch.int32, torch.int32, torch.int64)]
    kvq.kvq_slot_map(cuda_ints(held), start, ctx, dev, n_pages, *outs)
    rows = slot_map(held, want[1], want[2], want[0], n_pages, n_tokens)
    ref = np.array([(55, 55, 55) if r is None else r for r in rows])
    ref[:, 1] = ((ref[:, 1] + 2 ** 31) % 2 ** 32) - 2 ** 31  # positions wrap as int32
    for i in range(3):
        np.testing.assert_array_equal(outs[i].cpu().numpy(), ref[:, i])


@pytest.mark.parametrize("name", list(LENGTHS))
def test_tables_and_slots(name):
    held, new, pps, n_free, cursor = LENGTHS[name]
    # new tokens of refused requests count in seq_start as well; keep the batch's total small
    new = [n if n < 10 ** 6 else 11 for n in new]
    free = np.random.default_rng(2).permutation(n_free + 50)[:n_free].astype(np.int32)
    check_tables(np.array(held), np.array(new), pps, free, cursor)


@pytest.mark.parametrize("batch", [1, 31, 255, 256, 257, 1025])
def test_tables_and_slots_of_many_requests(batch):
    rng = np.random.default_rng(batch)
    held, new = rng.integers(0, 300, batch), rng.integers(0, 200, batch)
    need = int(np.sum(-(-(held + new) // PAGE) - -(-held // PAGE)))
    check_tables(held, new, 8, rng.permutation(need + 9).astype(np.int32), 4)


def test_rows_before_the_first_request_get_no_slot():
    """seq_start need not begin at 0: rows before it belong to no request, and an append must not see a slot there."""
    held, start, ctx = cuda_ints([70, 3]), cuda_ints([5, 7, 10]), cuda_ints([72, 6])
    table = cuda_ints([[4, 1], [0, 3]])
    outs = [cuda_ints(np.full(12, 55), t) for t in (torch.int32, torch.int32, torch.int64)]
    kvq.kvq_slot_map(held, start, ctx, table, 6, *outs)
    ids, pos, slots = (o.tolist() for o in outs)
    assert ids == [55] * 5 + [0, 0, 1, 1, 1] + [55] * 2
    assert pos == [55] * 5 + [70, 71, 3, 4, 5] + [55] * 2
    assert slots == [55] * 5 + [64 + 6, 64 + 7, 3, 4, 5] + [55] * 2


# ---- appends by slots

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", list(MODES))
def test_append_by_slots_stores_what_quantize_stores(name, dtype):
    """Shuffled tokens, one octet split between calls, a skipped token and a zero vector: the pool's bytes
    are those of kvq_quantize's appends, and no other byte changes."""
    cfg = make_cfg(4, 2, *MODES[name], rot_per_head=1)
    signs, S = signs_and_sketch(3, cfg)
    T, n_pages = 203, 9
    gen = torch.Generator(device="cuda").manual_seed(5)
    K, V = (torch.randn(2, T, 128, generator=gen, device="cuda").to(dtype) for _ in range(2))
    K[:, 17] = 0
    table = cuda_ints(np.random.default_rng(4).permutation(n_pages)[None, :5])
    a, b = (kvq.KvqCache(cfg, 1, 0, signs, S, block_table=table, n_pages=n_pages) for _ in range(2))
    for c in (a, b):
        c.arena[int(c.layout()[4]):].fill_(0x5A)
    for t in range(T):  # token by token: tile appends clear the rest of their tile
        a.quantize(K[None, :, t:t + 1].contiguous(), V[None, :, t:t + 1].contiguous(), seq_ids=[0])
    pos = torch.arange(T, device="cuda")
    slots = table[0].long()[pos // PAGE] * PAGE + pos % PAGE
    order = torch.randperm(T, generator=gen, device="cuda")
    for part in (order[:3], order[3:100], order[100:]):  # the whole again in order: overwrites with the same
        b.quantize_slots(K[:, part].transpose(0, 1).contiguous(), V[:, part].transpose(0, 1).contiguous(), slots[part])
    k2, v2 = K.transpose(0, 1).contiguous(), V.transpose(0, 1).contiguous()
    b.quantize_slots(k2, v2, slots)
    noise = torch.randn(3, 2, 128, device="cuda").to(dtype)
    b.quantize_slots(noise, noise, cuda_ints([-1, -7, -2 ** 62], torch.int64))
    assert kvq.kvq_cache_status(b.handle) == 0
    first = int(a.layout()[4])
    assert torch.equal(a.arena[first:], b.arena[first:])
    assert list(b.lengths()) == [0]
    b.quantize_slots(noise, noise, cuda_ints([-1, n_pages * PAGE, 2 ** 62], torch.int64))
    assert kvq.kvq_cache_status(b.handle) == 2
    assert torch.equal(a.arena[first:], b.arena[first:])
    a.close()
    b.close()


@pytest.mark.parametrize("tokens", [700, 1211, 1700])
@pytest.mark.parametrize("name", ["2q2q", "3q3", "11", "23q", "22", "1q2"])
def test_large_appends_store_what_small_ones_store(name, tokens):
    """One call, eager and captured, against calls of 100 tokens: every kernel of the append, sketches on both sides, one
    or none, and what follows it on the stream sees both sides."""
    cfg = make_cfg(8, 8, *MODES[name])
    signs, S = signs_and_sketch(4, cfg)
    n_pages = tokens // PAGE + 3
    gen = torch.Generator(device="cuda").manual_seed(6)
    K, V = (torch.randn(tokens, 8, 128, generator=gen, device="cuda").to(BF16) for _ in range(2))
    table = cuda_ints(np.random.default_rng(5).permutation(n_pages)[None, :])
    caches = [kvq.KvqCache(cfg, 1, 0, signs, S, block_table=table, n_pages=n_pages) for _ in range(3)]
    for c in caches:
        c.arena[int(c.layout()[4]):].fill_(0x5A)
    pos = torch.arange(tokens, device="cuda")
    slots = table[0].long()[pos // PAGE] * PAGE + pos % PAGE
    for i in range(0, tokens, 100):
        caches[0].quantize_slots(K[i:i + 100], V[i:i + 100], slots[i:i + 100])
    caches[1].quantize_slots(K, V, slots)
    seen = caches[1].arena.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caches[2].quantize_slots(K, V, slots)
    graph.replay()
    first = int(caches[0].layout()[4])
    for got in (seen, caches[1].arena, caches[2].arena):
        assert torch.equal(got[first:], caches[0].arena[first:])
    del graph
    for c in caches:
        c.close()


def test_lengths_set_without_an_append():
    """Decode over pages filled by slots, a sequence on another's pages, and a finished sequence's place."""
    cfg = make_cfg(4, 2, 2, True, 2, True)
    x = Batch(cfg, [130, 40], [3, 1], seed=6)
    q = x.q[:2].contiguous()
    x.cache.set_lengths([133, 41])
    assert list(x.cache.lengths()) == [133, 41]
    out = x.cache.decode(q)
    table = x.table.cpu().numpy()
    for b, T in enumerate((133, 41)):
        for hk in range(2):
            K, V = dequantised(x.cache, cfg, table, b, hk, T, x.signs, x.S)
            ref = causal_attention(q[b:b + 1, 2 * hk:2 * hk + 2].double().cpu().numpy(), K, V, T)
            assert_close(out[b:b + 1, 2 * hk:2 * hk + 2], ref, BF16)
    x.table[1, :2] = x.table[0, :2]                 # the first two pages of sequence 0
    x.cache.set_lengths(np.array([0, 128]))
    out = x.cache.decode(q)
    assert not out[0].any()
    K, V = dequantised(x.cache, cfg, table, 0, 0, 128, x.signs, x.S)
    assert_close(out[1:2, :2], causal_attention(q[1:2, :2].double().cpu().numpy(), K, V, 128), BF16)
    for lens, status in (([-1, 0], 1), ([0, 10 ** 6], 3)):
        with pytest.raises(kvq.KvqError) as e:
            x.cache.set_lengths(lens)
        assert e.value.status == status
    assert list(x.cache.lengths()) == [0, 128]
    x.cache.close()


# ---- attention of a ragged batch

RAGGED = [([0], [1]), ([63], [1]), ([0], [64]), ([64, 0, 200, 31, 7], [1, 1, 1, 0, 57]), ([500, 0, 129], [70, 33, 0]),
          ([1000, 3], [8, 140])]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", list(MODES))
def test_chunk_attention_modes(name, dtype):
    """Every code combination; the norms behind the tokens are NaN."""
    x = Batch(make_cfg(8, 2, *MODES[name], rot_per_head=1), [150, 0, 70], [9, 75, 40], dtype, seed=7)
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    assert kvq.kvq_cache_status(x.cache.handle) == 0
    assert out.dtype == dtype
    assert_close(out, x.reference(), dtype)
    x.cache.close()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("held,new", RAGGED)
def test_chunk_attention_lengths(held, new, group, dtype):
    for name in ("2q2q", "3q3"):
        x = Batch(make_cfg(2 * group, 2, *MODES[name]), held, new, dtype, seed=group)
        out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
        assert kvq.kvq_cache_status(x.cache.handle) == 0
        assert_close(out, x.reference(), dtype)
        x.cache.close()


@pytest.mark.parametrize("name", ["2q2q", "3q3", "11"])
def test_chunk_attention_of_long_chunks(name):
    """Several row tiles of a request and segments that end inside one; single tokens beside them."""
    x = Batch(make_cfg(8, 2, *MODES[name]), [900, 2500, 0, 3000], [300, 1, 517, 2], seed=8)
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    assert kvq.kvq_cache_status(x.cache.handle) == 0
    assert_close(out, x.reference(), BF16)
    x.cache.close()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_without_positions_and_rows_of_no_request(dtype):
    """A request whose context is shorter than its chunk: zeros for the rows before position 0. Rows before
    the first request and behind the last stay as they were."""
    x = Batch(make_cfg(4, 1, 2, True, 2, True), [0, 100], [40, 30], dtype, seed=9)
    q = torch.cat([x.q[:5], x.q, x.q[:6]])
    out = torch.full_like(q, 3.0)
    start, ctx = cuda_ints([5, 45, 75]), cuda_ints([12, 0])
    x.cache.chunk_attention(q, start, ctx, out=out)
    assert (out[:5] == 3).all() and (out[75:] == 3).all()
    assert not out[5:33].any() and not out[45:75].any()
    K, V = dequantised(x.cache, x.cfg, x.table.cpu().numpy(), 0, 0, 12, x.signs, x.S)
    assert_close(out[33:45], causal_attention(q[33:45].double().cpu().numpy(), K, V, 12), dtype)
    # lengths of the cache itself, and a batch in which no request has a token
    x.cache.set_lengths([40, 130])
    assert_close(x.cache.chunk_attention(x.q, cuda_ints([0, 40, 70])), x.reference(), dtype)
    out.fill_(3.0)
    x.cache.chunk_attention(q, cuda_ints([0, 0, 0]), out=out)
    assert (out == 3).all()
    x.cache.close()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e30])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_token_that_is_not_finite_reaches_only_the_rows_that_attend_to_it(where, value, dtype):
    """1e30 has an fp16 norm of infinity."""
    cfg = make_cfg(4, 1, 2, True, 2, True)
    new, bad = 100, 60
    kv = {n: torch.randn(new, 1, 128, device="cuda").to(dtype) for n in "kv"}
    kv[where][bad, 0, 3] = value
    x = Batch(cfg, [70], [new], dtype, seed=10, **kv)
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    rows = x.reference(torch.nan_to_num(x.q))[:bad]
    assert_close(out[:bad], rows, dtype)
    if where == "v" or value != value:
        assert out[bad:].isnan().all(-1).all()
    x.cache.close()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_a_query_that_is_not_finite_keeps_to_its_row(value):
    x = Batch(make_cfg(4, 2, 2, True, 2, True), [70, 30], [20, 9], seed=11)
    want = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    q = x.q.clone()
    q[13, 2, 5] = value
    out = x.cache.chunk_attention(q, x.seq_start, x.ctx_lens)
    assert out[13, 2].isnan().any()
    out[13, 2] = want[13, 2]
    assert torch.equal(out, want)
    x.cache.close()


@pytest.mark.parametrize("scale", [1e-3, 30.0, 4e3])
def test_large_and_small_queries_and_values(scale):
    """Rows whose softmax is uniform to within rounding, or one position's alone. Values up to the largest
    that the cache's fp16 norms hold: 4e3 sqrt(128) is 45e3 (a norm over 65504 is stored as infinity)."""
    cfg = make_cfg(4, 1, 3, False, 3, False)
    kv = {n: torch.randn(90, 1, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i)).to(BF16)
          for i, n in enumerate("kv")}
    kv["v"] = (kv["v"] * scale).to(BF16)
    x = Batch(cfg, [0], [90], seed=12, **kv)
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    assert_close(out, x.reference(), BF16)
    # with queries of another size the softmax picks one position: compared where its lead decides
    q = (x.q * 200).contiguous()
    out, ref = x.cache.chunk_attention(q, x.seq_start, x.ctx_lens), x.reference(q)
    K, _ = dequantised(x.cache, cfg, x.table.cpu().numpy(), 0, 0, 90, x.signs, x.S)
    logits = np.einsum("nhd,td->nht", q.double().cpu().numpy(), K) / np.sqrt(128)
    logits[np.broadcast_to(np.arange(90)[None, None] > np.arange(90)[:, None, None], logits.shape)] = -np.inf
    top = np.sort(logits, -1)
    # a logit's error: 3 roundings of 2^-11 of each product, at worst that of |q| |k|
    worst = 3 * 2.0 ** -11 * np.linalg.norm(q.double().cpu().numpy(), axis=-1) * np.linalg.norm(K, axis=-1).max() / np.sqrt(128)
    sure = top[..., -1] - top[..., -2] > 2 * worst + np.log(90 * 1e4)
    assert sure.mean() > 0.2
    assert_close(out[torch.tensor(sure)], ref[sure], BF16)
    x.cache.close()


def test_contiguous_cache_and_decode_agree():
    """A cache that is not paged; and one new token of every sequence is what decode computes."""
    cfg = make_cfg(8, 2, 2, True, 2, True)
    signs, S = signs_and_sketch(13, cfg)
    lens = [200, 64, 1]
    c = kvq.KvqCache(cfg, 3, 256, signs, S)
    for b, n in enumerate(lens):
        c.quantize(*(torch.randn(1, 2, n, 128, device="cuda").to(BF16) for _ in range(2)), seq_ids=[b])
    q = torch.randn(3, 8, 128, device="cuda").to(BF16)
    out = c.chunk_attention(q, cuda_ints([0, 1, 2, 3]))
    assert_close(out, c.decode(q).double().cpu().numpy(), BF16)
    for b, n in enumerate(lens):
        for hk in range(2):
            K, V = dequantised(c, cfg, None, b, hk, n, signs, S)
            assert_close(out[b:b + 1, 4 * hk:4 * hk + 4],
                         causal_attention(q[b:b + 1, 4 * hk:4 * hk + 4].double().cpu().numpy(), K, V, n), BF16)
    c.close()


def test_page_outside_the_pool_sets_status():
    x = Batch(make_cfg(4, 2, 2, True, 2, True), [200], [20], seed=14)
    x.table[0, 1] = 10 ** 6
    for q in (x.q, x.q.float()):
        out = x.cache.chunk_attention(q, x.seq_start, x.ctx_lens)
        torch.cuda.synchronize()
        assert out.shape == q.shape
    assert kvq.kvq_cache_status(x.cache.handle) == 2
    x.cache.close()


def test_refusals_of_a_live_cache():
    x = Batch(make_cfg(4, 2, 2, True, 2, True), [20], [5], seed=15)
    c = x.cache
    out = torch.empty_like(x.q)
    need = kvq.kvq_chunk_workspace_bytes(c.handle, BF16, 5)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    n = kvq.kvq_kernel_launches()
    for call, error in (
            (lambda: c.chunk_attention(x.q, x.seq_start, x.ctx_lens, out, ws[:-1]), kvq.KvqError),
            (lambda: c.chunk_attention(x.q, x.seq_start, x.ctx_lens, out.float()), TypeError),
            (lambda: c.chunk_attention(x.q, x.seq_start.long(), x.ctx_lens), TypeError),
            (lambda: c.chunk_attention(x.q.transpose(0, 1).contiguous().transpose(0, 1), x.seq_start), ValueError),
            (lambda: c.quantize_slots(x.q[:, :2].float().contiguous(), x.q[:, :2].contiguous(), x.seq_start.long()), TypeError),
            (lambda: c.quantize_slots(*(x.q[:, :2].contiguous(),) * 2, cuda_ints([0, 1, 2], torch.int64)), ValueError),
            (lambda: kvq.kvq_chunk_workspace_bytes(c.handle, F32, -1), kvq.KvqError),
            (lambda: kvq.kvq_chunk_workspace_bytes(c.handle, F32, (1 << 28) + 1), kvq.KvqError)):
        with pytest.raises(error):
            call()
    c.quantize_slots(x.q[:0, :2].contiguous(), x.q[:0, :2].contiguous(), cuda_ints([], torch.int64))  # no tokens
    assert kvq.kvq_kernel_launches() == n
    assert c.chunk_attention(x.q[:0], cuda_ints([0, 0])).shape == (0, 4, 128)
    other = kvq.KvqCache(kvq.make_cfg(128, 4, 2, sink_tokens=4, recent_tokens=60), 1, 128, x.signs, x.S)
    flat = kvq.KvqCache(x.cfg, 1, 128, x.signs, x.S)
    for fn in (lambda: other.chunk_attention(x.q, x.seq_start), lambda: other.set_lengths([0]),
               lambda: flat.quantize_slots(*(x.q[:, :2].contiguous(),) * 2, cuda_ints(range(5), torch.int64))):
        with pytest.raises(kvq.KvqError) as e:
            fn()
        assert e.value.status == 2
    for t in (c, other, flat):
        t.close()


def test_a_run_of_steps_captured_and_eager():
    """Prompts in chunks, single and speculated tokens, an idle request: the four calls of a step captured
    once and replayed with new lengths, against the same calls made eagerly on another stream."""
    cfg = make_cfg(8, 2, 2, True, 2, True)
    signs, S = signs_and_sketch(16, cfg)
    B, pps, n_pages, rows = 4, 6, 24, 200
    plan = [[120, 3, 0, 64], [60, 1, 1, 64], [1, 5, 1, 0], [1, 1, 130, 1]]
    gen = torch.Generator(device="cuda").manual_seed(16)
    data = [[torch.randn(rows, h, 128, generator=gen, device="cuda").to(BF16) for h in (2, 2, 8)] for _ in plan]
    results = []
    for captured in (True, False):
        table = torch.full((B, pps), -1, dtype=torch.int32, device="cuda")
        c = kvq.KvqCache(cfg, B, 0, signs, S, block_table=table, n_pages=n_pages)
        c.arena[int(c.layout()[4]):].fill_(0xFF)
        free, cursor = cuda_ints(np.random.default_rng(0).permutation(n_pages)), cuda_ints([0])
        held, new, taken = cuda_ints([0] * B), cuda_ints([0] * B), cuda_ints([0, 0])
        start, ctx = cuda_ints([0] * (B + 1)), cuda_ints([0] * B)
        slots = cuda_ints([-1] * rows, torch.int64)
        k, v, q = (torch.zeros_like(t) for t in data[0])
        out = torch.zeros_like(q)
        ws = torch.empty(kvq.kvq_chunk_workspace_bytes(c.handle, BF16, rows), dtype=torch.uint8, device="cuda")

        def step():
            slots.fill_(-1)
            kvq.kvq_extend_block_table(held, new, free, table, start, ctx, taken, cursor)
            cursor.add_(taken[:1])
            kvq.kvq_slot_map(held, start, ctx, table, n_pages, None, None, slots)
            c.quantize_slots(k, v, slots)
            c.chunk_attention(q, start, ctx, out, ws if captured else None)
            held.copy_(ctx)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        got = []
        with torch.cuda.stream(torch.cuda.current_stream() if captured else side):
            for n, (k1, v1, q1) in zip(plan, data):
                new.copy_(torch.tensor(n, dtype=torch.int32))
                k.copy_(k1), v.copy_(v1), q.copy_(q1)
                out.zero_()
                g.replay() if captured else step()
                got.append(out.clone())
        torch.cuda.synchronize()
        assert list(held.cpu()) == [sum(p[b] for p in plan) for b in range(B)]
        assert int(taken[1]) == 0 and kvq.kvq_cache_status(c.handle) == 0
        lens = np.zeros(B, dtype=int)
        for n, (_, _, q1), o in zip(plan, data, got):
            lens, at = lens + n, 0
            for b in range(B):
                for hk in range(2 if n[b] else 0):
                    K, V = dequantised(c, cfg, table.cpu().numpy(), b, hk, int(lens[b]), signs, S)
                    s = (slice(at, at + n[b]), slice(4 * hk, 4 * hk + 4))
                    assert_close(o[s], causal_attention(q1[s].double().cpu().numpy(), K, V, int(lens[b])), BF16)
                at += n[b]
            assert not o[at:].any()
        results.append(got)
        c.close()
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_two_graphs_and_two_streams_keep_apart():
    """Captured calls take their workspace from their graph's memory, eager ones from their stream's."""
    x = Batch(make_cfg(8, 2, 2, True, 2, True), [2000, 700], [40, 90], seed=17)
    ref = x.reference()
    qs = [x.q, x.q.flip(0).contiguous()]
    refs = [ref, x.reference(qs[1])]
    want = [x.cache.chunk_attention(q, x.seq_start, x.ctx_lens) for q in qs]
    for w, r in zip(want, refs):
        assert_close(w, r, BF16)
    graphs, outs = [], []
    for q in qs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(x.cache.chunk_attention(q, x.seq_start, x.ctx_lens))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        eager = []
        for g, s, q in zip(graphs, streams, qs):
            with torch.cuda.stream(s):
                g.replay()
                eager.append(x.cache.chunk_attention(q, x.seq_start, x.ctx_lens))
        torch.cuda.synchronize()
        for o, e, w in zip(outs, eager, want):
            assert torch.equal(o, w) and torch.equal(e, w)
    x.cache.close()


def test_the_same_call_gives_the_same_bits():
    x = Batch(make_cfg(8, 1, 3, True, 3, False), [5000], [130], seed=18)
    first = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    for _ in range(4):
        assert torch.equal(x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens), first)
    x.cache.close()


@pytest.mark.parametrize("name,group", [("2q2q", 4), ("3q3", 8), ("22", 1), ("23q", 2)])
@pytest.mark.parametrize("rows", [24, 32, 40, 128, 136, 256, 264, 512, 520, 1032])
def test_row_counts_around_the_tiles(rows, name, group):
    """The last rows of the narrow kernel's tile, of a CTA's half, of a tile and of a pair of them, and one token
    more: beside a request of a single token."""
    x = Batch(make_cfg(group, 1, *MODES[name]), [77, 300], [rows // group, 1], seed=rows)
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    assert kvq.kvq_cache_status(x.cache.handle) == 0
    assert_close(out, x.reference(), BF16)
    x.cache.close()


@pytest.mark.parametrize("batch", [255, 257, 520])
def test_chunk_attention_of_many_requests(batch):
    """More requests than a block of the plan has threads, some without tokens, some with a wide tile."""
    rng = np.random.default_rng(batch)
    new = rng.integers(0, 4, batch)
    new[[5, batch - 2]] = [50, 70]
    x = Batch(make_cfg(2, 1, 2, True, 2, True), rng.integers(0, 150, batch), new, seed=batch)
    for q in (x.q, x.q.float()):
        assert_close(x.cache.chunk_attention(q, x.seq_start, x.ctx_lens), x.reference(q), q.dtype)
    x.cache.close()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("new", [3, 30, 200])
@pytest.mark.parametrize("name", ["2q2q", "33"])
def test_maxima_that_grow_along_the_context(name, new, dtype):
    """Keys that point more and more along the queries: a row's maximum grows by far more than the lag that its
    reference may have, in every part of a page and many times over, so that what was summed before has to
    follow. At the end one position holds nearly all of the weight; before, several."""
    cfg = make_cfg(4, 1, *MODES[name])
    held = 700
    gen = torch.Generator(device="cuda").manual_seed(3)
    way = torch.randn(128, generator=gen, device="cuda")
    n = held + new
    size = torch.linspace(0.02, 3.0, n, device="cuda")[:, None, None]
    k = (way * size + 0.3 * torch.randn(n, 1, 128, generator=gen, device="cuda")).to(dtype)
    v = torch.randn(n, 1, 128, generator=gen, device="cuda").to(dtype)
    x = Batch(cfg, [0], [n], dtype, seed=21, k=k, v=v)
    q = (way * 0.8 + 0.3 * torch.randn(new, 4, 128, generator=gen, device="cuda")).to(dtype)
    x.new = np.array([new])
    out = x.cache.chunk_attention(q, cuda_ints([0, new]), x.ctx_lens)
    ref = x.reference(q)
    # logits up to 0.8 * 3 * |way|^2 / sqrt(128), about 27: an operand's half step of 2^-11 on each product, three of them
    # and of either sign, moves one by up to 3 * 2^-11 * 27 / sqrt(128) * 4 (four sigma) = 0.014, the weights that
    # share a row by as much of their size
    top = np.abs(ref).max(-1, keepdims=True)
    tol = 2e-4 * top if dtype == F32 else 0.03 * top + 2.0 ** -8 * np.abs(ref)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    x.cache.close()


@pytest.mark.parametrize("name,group", [("2q2q", 4), ("3q3", 8), ("22", 1), ("23q", 2)])
@pytest.mark.parametrize("rows", [40, 48, 56, 64, 72])
def test_narrow_tiles_of_more_than_32_rows(rows, name, group):
    """Tiles of 33 to 64 rows in one call with smaller ones, over contexts that end in the first or the second page of a
    step and that several CTAs share; 72 rows go to the wide kernel, the rest of the call stays."""
    x = Batch(make_cfg(2 * group, 2, *MODES[name]), [77, 300, 1500, 2, 0],
              [rows // group, 1, 40 // group, 32 // group, 48 // group], seed=rows)
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    assert kvq.kvq_cache_status(x.cache.handle) == 0
    assert_close(out, x.reference(), BF16)
    assert torch.equal(x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens), out)
    x.cache.close()


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("bad", [3, 12])
def test_a_token_that_is_not_finite_in_a_tile_of_64_rows(bad, where, value):
    """Rows of either half of the tile before the token, behind it, and another request's: only those behind change."""
    cfg = make_cfg(4, 1, 2, True, 2, True)
    kv = {n: torch.randn(16 + 3, 1, 128, device="cuda").to(BF16) for n in "kv"}
    kv[where][bad, 0, 3] = value
    x = Batch(cfg, [120, 30], [16, 3], seed=23, **kv)
    out, ref = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens), x.reference()
    assert_close(out[:bad], ref[:bad], BF16)
    assert_close(out[16:], ref[16:], BF16)
    if where == "v" or value != value:
        assert out[bad:16].isnan().all(-1).all()
    x.cache.close()


@pytest.mark.parametrize("name", ["2q2q", "33"])
def test_maxima_that_grow_in_a_tile_of_64_rows(name):
    test_maxima_that_grow_along_the_context(name, 13, BF16)


def test_long_context_of_one_token():
    """A single token over a context that every CTA of the narrow kernel shares."""
    x = Batch(make_cfg(4, 1, 2, True, 2, True), [40000], [1], seed=22)
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    x.cache.set_lengths([40001])
    ref = x.cache.decode(x.q)
    top = ref.abs().amax(-1, keepdim=True)
    # decode is within 2e-3 of a row's largest entry (its own tests); this call as in assert_close
    assert ((out.double() - ref.double()).abs() <= (7e-3 * top + 2.0 ** -8 * ref.abs())).all()
    x.cache.close()


def test_on_a_stream_given_by_name():
    x = Batch(make_cfg(8, 2, 2, True, 2, True), [600, 3], [40, 2], seed=23)
    want = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(x.q)
    x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    assert len(x.cache.chunk_workspaces) == 2
    x.cache.close()
