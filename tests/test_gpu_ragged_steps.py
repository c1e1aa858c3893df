"""Steps of the ragged serving path one after the other on the GPU: buffers that are kept, requests that are refused,
appends of every kernel, what calls share."""
import threading

import numpy as np
import pytest
import torch

import bit_kv_cache_seeded_b200 as kvq
from tests._ragged import PAGE, Batch, assert_close, causal_attention, cuda_ints, dequantised, make_cfg, signs_and_sketch

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    kvq.load()


class Server:
    """A server's step, on buffers of a fixed size that are never filled between steps."""

    def __init__(self, cfg, batch, pages_per_seq, n_pages, rows, dtype=BF16, seed=0):
        self.cfg, self.n_pages = cfg, n_pages
        self.signs, self.S = signs_and_sketch(seed, cfg)
        self.table = torch.full((batch, pages_per_seq), -1, dtype=torch.int32, device="cuda")
        self.cache = kvq.KvqCache(cfg, batch, 0, self.signs, self.S, block_table=self.table, n_pages=n_pages)
        self.first = int(self.cache.layout()[4])
        self.cache.arena[self.first:].fill_(0x5A)
        self.free, self.cursor = cuda_ints(np.random.default_rng(seed).permutation(n_pages)), cuda_ints([0])
        self.held, self.new = cuda_ints([0] * batch), cuda_ints([0] * batch)
        self.start, self.ctx, self.taken = cuda_ints([0] * (batch + 1)), cuda_ints([0] * batch), cuda_ints([0, 0])
        self.slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        self.k, self.v = (torch.zeros(rows, cfg.n_kv_heads, 128, dtype=dtype, device="cuda") for _ in range(2))
        self.q = torch.zeros(rows, cfg.n_q_heads, 128, dtype=dtype, device="cuda")
        self.gen = torch.Generator(device="cuda").manual_seed(seed)

    def inputs(self, new):
        self.new.copy_(torch.tensor(new, dtype=torch.int32))
        for t in (self.k, self.v, self.q):
            t.copy_(torch.randn(t.shape, generator=self.gen, device="cuda"))

    def append(self):
        kvq.kvq_extend_block_table(self.held, self.new, self.free, self.table, self.start, self.ctx, self.taken, self.cursor)
        kvq.kvq_slot_map(self.held, self.start, self.ctx, self.table, self.n_pages, None, None, self.slots)
        self.cache.quantize_slots(self.k, self.v, self.slots, seq_start=self.start)

    def advance(self):
        self.cursor.add_(self.taken[:1])
        self.held.copy_(self.ctx)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [160, 1300])
@pytest.mark.parametrize("name", [(2, True, 2, True), (1, False, 1, False), (3, True, 3, False)])
def test_a_short_step_after_a_long_one_leaves_the_rest_of_the_pool(name, rows, dtype):
    """The slots behind a step's tokens are still the long step's; they may also be anything else. The pool is that of an
    append of the step's tokens alone."""
    s = Server(make_cfg(4, 4, *name), 3, rows // PAGE + 2, rows // PAGE + 6, rows, dtype)
    s.inputs([rows - 70, 0, 70])
    s.append()
    s.advance()
    alone = kvq.KvqCache(s.cfg, 3, 0, s.signs, s.S, block_table=s.table, n_pages=s.n_pages)
    for new, junk in (([1, 1, 0], False), ([0, 0, 0], False), ([0, 2, 3], True)):
        alone.arena[s.first:] = s.cache.arena[s.first:]
        s.inputs(new)
        if junk:
            s.slots.copy_(torch.randint(-2 ** 62, 2 ** 62, s.slots.shape, device="cuda"))
            s.slots[-40:] = torch.arange(40, device="cuda")
        s.append()
        s.advance()
        n = sum(new)
        alone.quantize_slots(s.k[:n], s.v[:n], s.slots[:n])
        assert torch.equal(alone.arena[s.first:], s.cache.arena[s.first:])
    assert kvq.kvq_cache_status(s.cache.handle) == 0
    alone.close()
    s.cache.close()


@pytest.mark.parametrize("name", [(2, True, 2, True), (1, False, 1, False), (3, True, 3, False)])
@pytest.mark.parametrize("tokens", [40, 700, 1700])
def test_rows_of_requests_alone_are_appended(name, tokens):
    """Requests that begin behind the first row and end before the last: the pool's bytes are those of an append of
    their rows by themselves."""
    cfg = make_cfg(8, 8, *name)
    signs, S = signs_and_sketch(2, cfg)
    n_pages = tokens // PAGE + 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    K, V = (torch.randn(tokens, 8, 128, generator=gen, device="cuda").to(BF16) for _ in range(2))
    slots = torch.randperm(n_pages * PAGE, generator=gen, device="cuda")[:tokens]
    table = cuda_ints(np.full((2, n_pages), -1))
    caches = [kvq.KvqCache(cfg, 2, 0, signs, S, block_table=table, n_pages=n_pages) for _ in range(2)]
    for c in caches:
        c.arena[int(c.layout()[4]):].fill_(0x5A)
    a, b = 5, tokens - 9
    caches[0].quantize_slots(K, V, slots, seq_start=cuda_ints([a, a + 7, b]))
    alone = torch.full_like(slots, -1)
    alone[a:b] = slots[a:b]
    caches[1].quantize_slots(K, V, alone)
    first = int(caches[0].layout()[4])
    assert torch.equal(caches[0].arena[first:], caches[1].arena[first:])
    for start in ([0, 0, 0], [tokens, tokens, tokens], [-5, -3, -1], [9, 9, 2]):  # no row of a request
        caches[0].quantize_slots(K.flip(0).contiguous(), V, slots, seq_start=cuda_ints(start))
    assert torch.equal(caches[0].arena[first:], caches[1].arena[first:])
    caches[0].quantize_slots(K, V, slots, seq_start=cuda_ints([-3, 0, tokens + 100]))  # all of them
    caches[1].quantize_slots(K, V, slots)
    assert torch.equal(caches[0].arena[first:], caches[1].arena[first:])
    for c in caches:
        c.close()


# ---- refused requests

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("name", [(2, True, 2, True), (3, True, 3, False)])
def test_a_refused_request_between_granted_ones(name, dtype):
    """The four calls of a step that refuses a request of one, of a few and of many tokens: nothing of it is appended, its
    rows get zeros, and the others get what they get without it. The next step goes on from the lengths that are left."""
    cfg = make_cfg(4, 2, *name)
    s = Server(cfg, 5, 6, 16, 400, dtype)
    s.inputs([100, 40, 200, 10, 0])
    s.append()
    s.advance()
    for new, over in (([20, 120, 3, 70, 1], 1), ([6, 10, 250, 0, 0], 2), ([1, 2, 4, 400, 3], 3), ([5, -1, 5, 5, 5], 1)):
        total = sum(max(n, 0) for n in new)
        if over == 1 and new[1] > 0:      # want of pages: the free list ends behind the request's first
            s.free = s.free[:int(s.cursor) + 1].contiguous()
        if total > s.slots.numel():
            s.slots = torch.empty(total, dtype=torch.int64, device="cuda")
            s.k, s.v = (torch.empty(total, 2, 128, dtype=dtype, device="cuda") for _ in range(2))
            s.q = torch.empty(total, 4, 128, dtype=dtype, device="cuda")
        s.inputs(new)
        held = s.held.tolist()
        s.append()
        granted = [c == h + max(n, 0) and n >= 0 for c, h, n in zip(s.ctx.tolist(), held, new)]
        assert not granted[over] and int(s.taken[1]) == granted.count(False)
        out = s.cache.chunk_attention(s.q, s.start, s.ctx, out=torch.full_like(s.q, 3.0), held=s.held)
        ref, at = np.zeros((total, 4, 128)), 0
        for b, n in enumerate(max(n, 0) for n in new):
            for hk in range(2 if granted[b] and n else 0):
                K, V = dequantised(s.cache, cfg, s.table.cpu().numpy(), b, hk, held[b] + n, s.signs, s.S)
                ref[at:at + n, 2 * hk:2 * hk + 2] = causal_attention(s.q[at:at + n, 2 * hk:2 * hk + 2].double().cpu().numpy(),
                                                                     K, V, held[b] + n)
            if not granted[b]:
                assert not out[at:at + n].any()
            at += n
        assert_close(out[:total], ref, dtype)
        assert (out[total:] == 3).all()
        s.advance()
        assert s.held.tolist() == [h + n if g else h for h, n, g in zip(held, new, granted)]
    assert kvq.kvq_cache_status(s.cache.handle) == 0
    s.cache.close()


# ---- streams and threads

def test_out_on_a_stream_given_by_name():
    """The result is the given stream's memory; what is pending on the current stream does not reach it."""
    x = Batch(make_cfg(8, 2, 2, True, 2, True), [600, 3], [40, 2], seed=24)
    want = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = torch.full_like(want, 3.0)
    del old                                     # its memory is the next of the current stream's
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens, stream=s)
    of = {seg["address"]: (seg["total_size"], seg["stream"]) for seg in torch.cuda.memory_snapshot()}
    at = [stream for base, (size, stream) in of.items() if base <= out.data_ptr() < base + size]
    assert at == [s.cuda_stream]
    s.synchronize()
    assert torch.equal(out, want)
    x.cache.close()


def test_threads_on_one_stream():
    """Calls of four threads on the default stream, small and large, fp32 and bf16, without workspaces of their own."""
    x = Batch(make_cfg(8, 2, 2, True, 2, True), [2000, 3, 70], [40, 2, 90], seed=25)
    qs = [x.q, x.q.flip(0).contiguous(), x.q.float(), (0.5 * x.q).contiguous()]
    want = [x.cache.chunk_attention(q, x.seq_start, x.ctx_lens) for q in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]

    def work(i):
        for _ in range(20):
            got[i].append(x.cache.chunk_attention(qs[i], x.seq_start, x.ctx_lens))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(qs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert len(outs) == 20 and all(torch.equal(o, w) for o in outs)
    assert len(x.cache.chunk_workspaces) == 1
    x.cache.close()


# ---- values that are not finite, in many short segments

@pytest.mark.parametrize("name", [(2, True, 2, True), (2, False, 3, True), (3, True, 3, False), (1, False, 1, False)])
def test_values_that_are_not_finite_in_many_one_page_segments(name):
    """More one-page segments a pair of CTAs than its ring of markers has slots, several of them with a token that is not
    finite, at its first, a middle or its last position: the rows from that token on are NaN, and no other."""
    B, group, heads = 700, 4, 4                    # 2800 row tiles of 72 to 256 rows on 74 pairs: 37 each
    rng = np.random.default_rng(26)
    new = rng.integers(18, 65, B)
    start = np.concatenate([[0], np.cumsum(new)])
    gen = torch.Generator(device="cuda").manual_seed(26)
    v = torch.randn(int(start[-1]), heads, 128, generator=gen, device="cuda").to(BF16)
    bad = {}
    for b in rng.choice(B, 160, replace=False):
        i, h = int(rng.choice([0, new[b] // 2, new[b] - 1])), int(rng.integers(heads))
        v[start[b] + i, h, 5] = float(rng.choice([np.nan, np.inf]))
        bad[b] = (i, h)
    cfg = make_cfg(group * heads, heads, *name)
    x = Batch(cfg, [0] * B, new, seed=26, v=v)
    for _ in range(3):
        out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
        nan = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
        for b, (i, h) in bad.items():
            nan[start[b] + i:start[b + 1], h * group:(h + 1) * group] = True
        assert torch.equal(out.isnan().all(-1), nan) and torch.equal(out.isnan().any(-1), nan)
    # the finite ones of some requests, with and without a bad token in another head
    table = x.table.cpu().numpy()
    for b in [*list(bad)[:6], 0, 349, B - 1]:
        for h in range(heads):
            upto = bad[b][0] if b in bad and bad[b][1] == h else int(new[b])
            K, V = dequantised(x.cache, cfg, table, b, h, int(new[b]), x.signs, x.S)
            rows = (slice(start[b], start[b] + upto), slice(h * group, (h + 1) * group))
            if upto:
                assert_close(out[rows], causal_attention(x.q[rows].double().cpu().numpy(), K[:upto], V[:upto], upto), BF16)
    assert kvq.kvq_cache_status(x.cache.handle) == 0
    x.cache.close()


@pytest.mark.parametrize("n_free", [600000, 200000])
def test_block_tables_of_the_most_requests(n_free):
    """2^20 requests of up to 138 tokens that need 229000 pages: enough free pages, and too few."""
    B, pps = 1 << 20, 2
    gen = torch.Generator(device="cuda").manual_seed(27)
    held = torch.randint(0, 100, (B,), generator=gen, device="cuda", dtype=torch.int32)
    new = torch.randint(0, 40, (B,), generator=gen, device="cuda", dtype=torch.int32)
    free = torch.randperm(n_free, generator=gen, device="cuda").int()
    table, cursor = torch.full((B, pps), -7, dtype=torch.int32, device="cuda"), cuda_ints([5])
    start, ctx, taken = cuda_ints(np.zeros(B + 1)), cuda_ints(np.zeros(B)), cuda_ints([0, 0])
    kvq.kvq_extend_block_table(held, new, free, table, start, ctx, taken, cursor)
    h, n = held.long(), new.long()
    fits = h + n <= pps * PAGE
    p0, p1 = (h + PAGE - 1) // PAGE, (h + n + PAGE - 1) // PAGE
    need = torch.where(fits, p1 - p0, 0)
    end = need.cumsum(0)
    ok = fits & ((need == 0) | (end <= free.numel() - 5))
    assert bool((~ok & fits).any()) == (n_free == 200000)
    page = torch.arange(pps, device="cuda")
    mine = ok[:, None] & (page >= p0[:, None]) & (page < p1[:, None])
    at = (5 + (end - need - p0)[:, None] + page).clamp(0, free.numel() - 1)
    assert torch.equal(table, torch.where(mine, free[at], -7))
    assert torch.equal(start[1:].long(), n.cumsum(0)) and int(start[0]) == 0
    assert torch.equal(ctx.long(), torch.where(ok, h + n, h))
    assert taken.tolist() == [int((need * ok).sum()), int((~ok).sum())]


def test_chunk_attention_of_the_most_heads():
    """A row tile of 512 tokens and 8192 heads ends just below 2^31 bytes of queries; more heads are refused."""
    cfg = make_cfg(8192, 8192, 3, True, 3, False)
    x = Batch(cfg, [0], [512], seed=28)
    out = x.cache.chunk_attention(x.q, x.seq_start, x.ctx_lens)
    table = x.table.cpu().numpy()
    for h in (0, 8191):
        K, V = dequantised(x.cache, cfg, table, 0, h, 512, x.signs, x.S)
        assert_close(out[:, h:h + 1], causal_attention(x.q[:, h:h + 1].double().cpu().numpy(), K, V, 512), BF16)
    assert kvq.kvq_cache_status(x.cache.handle) == 0
    x.cache.close()
    more = kvq.KvqCache(make_cfg(8193, 8193, 3, True, 3, False), 1, 64, x.signs, x.S)
    n = kvq.kvq_kernel_launches()
    q, ws = torch.zeros(65, 8193, 128, dtype=BF16, device="cuda"), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for call in (lambda: more.chunk_attention(q, cuda_ints([0, 65])), lambda: more.chunk_attention(q, cuda_ints([0, 65]), workspace=ws)):
        with pytest.raises(kvq.KvqError) as e:
            call()
        assert e.value.status == 2
    assert kvq.kvq_kernel_launches() == n
    more.close()


# ---- appends of blocks of 32 tokens

@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("tokens", [700, 1211, 1700])
@pytest.mark.parametrize("name", [(2, True, 2, True), (3, True, 3, False), (2, False, 3, True), (2, False, 2, False),
                                  (1, False, 1, False), (1, True, 2, False)])
def test_large_appends_in_any_order(name, tokens, dtype):
    """Shuffled slots, runs that begin inside an octet, skipped tokens and slots past the pool inside a block, a zero vector,
    a rotation per head: the bytes of calls of 100 tokens, whose kernel is compared with kvq_quantize."""
    cfg = make_cfg(8, 8, *name, rot_per_head=1)
    signs, S = signs_and_sketch(29, cfg)
    n_pages = tokens // PAGE + 4
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    K, V = (torch.randn(tokens, 8, 128, generator=gen, device="cuda").to(dtype) for _ in range(2))
    K[33], V[tokens // 2] = 0, 0
    table = cuda_ints(np.full((1, n_pages), -1))
    run = 5 + torch.arange(tokens, device="cuda")
    holes = run.clone()
    holes[3::7] = -torch.arange(1, len(holes[3::7]) + 1, device="cuda")
    holes[40:45] = n_pages * PAGE + torch.arange(5, device="cuda")
    holes[tokens - 3] = 2 ** 62
    shuffled = torch.randperm(n_pages * PAGE, generator=gen, device="cuda")[:tokens]
    shuffled[50] = -1
    turned = torch.where(run // 8 % 2 == 0, run ^ 7, run)  # octets backwards, every other one
    turned[turned >= 5 + tokens] = -2
    for slots, status in ((run, 0), (run.flip(0).contiguous(), 0), (shuffled, 0), (turned, 0), (holes, 2)):
        large, small = (kvq.KvqCache(cfg, 1, 0, signs, S, block_table=table, n_pages=n_pages) for _ in range(2))
        first = int(large.layout()[4])
        for c in (large, small):
            c.arena[first:].fill_(0x5A)
        large.quantize_slots(K, V, slots)
        for i in range(0, tokens, 100):
            small.quantize_slots(K[i:i + 100], V[i:i + 100], slots[i:i + 100])
        assert torch.equal(large.arena[first:], small.arena[first:])
        assert kvq.kvq_cache_status(large.handle) == status
        large.close()
        small.close()


@pytest.mark.parametrize("name", [(2, True, 2, True), (3, True, 3, False), (1, True, 2, False)])
@pytest.mark.parametrize("tokens", [100, 700])
def test_a_slot_named_twice_leaves_its_neighbours(tokens, name):
    """Within a block of tokens, and between blocks far apart; the other tokens' codes, signs and norms are those of a call
    without the second mention."""
    cfg = make_cfg(8, 8, *name)
    signs, S = signs_and_sketch(30, cfg)
    n_pages = tokens // PAGE + 2
    gen = torch.Generator(device="cuda").manual_seed(30)
    K, V = (torch.randn(tokens, 8, 128, generator=gen, device="cuda").to(BF16) for _ in range(2))
    table = cuda_ints(np.arange(n_pages)[None])
    twice, once = (kvq.KvqCache(cfg, 1, 0, signs, S, block_table=table, n_pages=n_pages) for _ in range(2))
    for c in (twice, once):
        c.arena[int(c.layout()[4]):].zero_()
    slots = torch.arange(tokens, device="cuda")
    named = slots.clone()
    again = {4: 3, 20: 60, tokens - 1: 8, tokens - 9: 9, 33: 33 - 16}   # row: the slot it names too
    for row, slot in again.items():
        named[row] = slot
        slots[row] = -1
    twice.quantize_slots(K, V, named)
    once.quantize_slots(K, V, slots)
    keep = [t for t in range(tokens) if t not in again and t not in again.values()]
    for h in (0, 7):
        for a, b in zip(dequantised(twice, cfg, table.cpu().numpy(), 0, h, tokens, signs, S),
                        dequantised(once, cfg, table.cpu().numpy(), 0, h, tokens, signs, S)):
            np.testing.assert_array_equal(a[keep], b[keep])
    assert kvq.kvq_cache_status(twice.handle) == 0
    twice.close()
    once.close()


def test_pages_behind_4_gib_of_a_pool():
    """The same tokens on the first pages of a small pool and on the last pages of one of 4.9 GB a side: the same bits."""
    cfg = make_cfg(16, 8, 3, True, 3, True)
    signs, S = signs_and_sketch(31, cfg)
    held, new = [500, 70, 0], [90, 3, 200]
    tokens = sum(held) + sum(new)
    gen = torch.Generator(device="cuda").manual_seed(31)
    K, V = (torch.randn(tokens, 8, 128, generator=gen, device="cuda").to(BF16) for _ in range(2))
    q = torch.randn(sum(new), 16, 128, generator=gen, device="cuda")
    results = []
    for n_pages, free in ((20, np.arange(20)), (140000, 139999 - np.arange(20))):
        table = torch.full((3, 10), -1, dtype=torch.int32, device="cuda")
        c = kvq.KvqCache(cfg, 3, 0, signs, S, block_table=table, n_pages=n_pages)
        info = c.layout()
        assert n_pages == 20 or int(info[1]) * 16 * (n_pages - 20) > 2 ** 32
        start, ctx, taken, cursor, at, got = cuda_ints([0] * 4), cuda_ints([0] * 3), cuda_ints([0, 0]), cuda_ints([0]), 0, []
        for have, more in (([0] * 3, held), (held, new)):
            n = sum(more)
            slots = torch.empty(n, dtype=torch.int64, device="cuda")
            kvq.kvq_extend_block_table(cuda_ints(have), cuda_ints(more), cuda_ints(free), table, start, ctx, taken, cursor)
            kvq.kvq_slot_map(cuda_ints(have), start, ctx, table, n_pages, None, None, slots)
            c.quantize_slots(K[at:at + n], V[at:at + n], slots, seq_start=start)
            cursor += taken[:1]
            at += n
        assert int(taken[1]) == 0
        for dtype in (BF16, F32):
            got.append(c.chunk_attention(q.to(dtype), start, ctx, held=cuda_ints(held)))
        c.set_lengths([h + n for h, n in zip(held, new)])
        got.append(c.decode(q[:3].contiguous()))
        assert kvq.kvq_cache_status(c.handle) == 0
        results.append(got)
        c.close()
        del c
    for a, b in zip(*results):
        assert a.isfinite().all() and torch.equal(a, b)


def test_captured_steps_without_a_fill_and_with_refusals():
    """The whole step captured once and replayed with long steps, short ones, empty ones and refused requests, against the
    same steps made eagerly: the same pools, lengths and results."""
    cfg, rows = make_cfg(8, 2, 2, True, 2, True), 200
    plan = [[120, 3, 0, 64], [1, 1, 1, 1], [0, 0, 0, 0], [5, 190, 1, 0], [1, 0, 130, 60], [-4, 2, 1, 1], [60, 60, 0, 70]]
    results = []
    for captured in (True, False):
        s = Server(cfg, 4, 4, 9, rows, seed=32)
        out, got = torch.zeros_like(s.q), []

        def step():
            s.append()
            s.cache.chunk_attention(s.q, s.start, s.ctx, out=out, held=s.held)
            s.advance()
        if captured:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step()
        for new in plan:
            s.inputs(new)
            out.fill_(3.0)
            g.replay() if captured else step()
            got += [out.clone(), s.held.clone(), s.taken.clone(), s.cache.arena[s.first:].clone()]
        assert kvq.kvq_cache_status(s.cache.handle) == 0
        results.append(got)
        if captured:
            del g
        s.cache.close()
    for a, b in zip(*results):
        assert torch.equal(a, b)
    refused = [int(t[1]) for t in results[0][2::4]]
    assert refused[:3] == [0, 0, 0] and sum(refused) >= 3
    total = [min(rows, sum(max(n, 0) for n in new)) for new in plan]
    assert all((o[n:] == 3).all() for o, n in zip(results[0][::4], total))
