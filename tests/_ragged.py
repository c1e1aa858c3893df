"""Plain 64-bit forms of the ragged serving path's operators, for its tests."""
import math

import numpy as np
import torch

import bit_kv_cache_seeded_b200 as kvq
from oracle import attention, tables
from tests._cache_reader import bits_from_words, codes_from_planes, side_fields

PAGE = 64


def make_cfg(hq, hkv, kb, kq, vb, vq, **kw):
    mode = lambda b, s: "lm_qjl" if s else ("sign1" if b == 1 else "lm")  # noqa: E731
    return kvq.make_cfg(128, hq, hkv, mode(kb, kq), mode(vb, vq), kb, vb, 128 if kq or vq else 0, **kw)


def signs_and_sketch(seed, cfg):
    rng = np.random.default_rng(seed)
    n = cfg.n_kv_heads if cfg.rot_per_head else 1
    signs = (rng.integers(0, 2, (n, 128)) * 2 - 1).astype(np.int8)
    return (signs if cfg.rot_per_head else signs[0]), rng.standard_normal((128, 128)).astype(np.float32)


def extend_block_table(held, new, free, cursor, table):
    """Plain form of kvq_extend_block_table: table (a copy, extended), seq_start, ctx_lens, taken."""
    table, pps = table.copy(), table.shape[1]
    start, ctx, asked, given, refused = [0], [], 0, 0, 0
    room = len(free) - cursor if 0 <= cursor <= len(free) else -1
    for b, (h, n) in enumerate(zip(held.tolist(), new.tolist())):
        start.append(start[-1] + max(n, 0))
        ok, need = h >= 0 and n >= 0 and h + n <= pps * PAGE, 0
        p0 = -(-h // PAGE)
        if ok:
            need = -(-(h + n) // PAGE) - p0
            at, asked = asked, asked + need
            ok = need == 0 or asked <= room
        if ok and need:
            table[b, p0:p0 + need] = free[cursor + at:cursor + at + need]
        given += need if ok else 0
        refused += 0 if ok else 1
        ctx.append(h + n if ok else min(max(h, 0), pps * PAGE))
    return table, np.array(start), np.array(ctx), np.array([given, refused])


def slot_map(held, start, ctx, table, n_pages, n_tokens):
    """Plain form of kvq_slot_map; None in rows behind the last request."""
    rows = [None] * n_tokens
    for b in range(len(held)):
        n = int(start[b + 1] - start[b])
        for i in range(n):
            t, pos, slot = int(start[b]) + i, int(held[b]) + i, -1
            if t >= n_tokens:
                break
            if int(held[b]) + n == int(ctx[b]) and 0 <= pos < table.shape[1] * PAGE:
                page = int(table[b, pos // PAGE])
                slot = page * PAGE + pos % PAGE if 0 <= page < n_pages else -1
            rows[t] = (b, pos, slot)
    return rows


def dequantised(cache, cfg, table, b, hk, T, signs, S):
    """K, V [T, 128] fp64 of one (sequence, kv-head), read from the arena's bytes. table: host array, or None."""
    arena, info = cache.arena.cpu().numpy(), cache.layout()
    sides = []
    for side, bits in ((0, cfg.k_bits), (1, cfg.v_bits)):
        tb, region = int(info[1 + side]), int(info[4 + side])
        nt = -(-T // 32)
        if table is None:
            first = (b * cfg.n_kv_heads + hk) * int(info[3])
            index = [first + t for t in range(nt)]
        else:
            index = [(int(table[b, t // 2]) * cfg.n_kv_heads + hk) * 2 + t % 2 for t in range(nt)]
        tiles = np.concatenate([arena[region + i * tb:region + (i + 1) * tb] for i in index] or [np.zeros(0, np.uint8)])
        one = np.array(info, copy=True)
        one[3], one[4 + side] = nt, 0
        planes, sketch, n16, g16 = side_fields(tiles, one, side, 0, T)
        z = None if sketch is None else bits_from_words(sketch)
        cent, _ = tables.lloyd_max_tables_f32(bits)
        sg = signs[hk] if np.ndim(signs) == 2 else signs
        sides.append(attention.dequantize_many(codes_from_planes(planes), n16, cent, sg, g16, z, S if z is not None else None))
    return sides


def causal_attention(q, K, V, ctx, scale=1.0 / math.sqrt(128)):
    """q [n, g, 128] of the last n of ctx tokens; row i attends to positions <= ctx - n + i. Zeros where none."""
    n, g, d = q.shape
    out = np.zeros((n, g, d))
    for i in range(n):
        T = ctx - n + i + 1
        if T > 0:
            logits = scale * (q[i] @ K[:T].T)
            w = np.exp(logits - logits.max(1, keepdims=True))
            out[i] = (w @ V[:T]) / w.sum(1, keepdims=True)
    return out


def cuda_ints(x, dtype=torch.int32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


class Batch:
    """A paged cache filled through the ragged path: tokens held, then new ones, on shuffled pages."""

    def __init__(self, cfg, held, new, dtype=torch.bfloat16, seed=0, spare=2, k=None, v=None):
        rng = np.random.default_rng(seed)
        self.cfg, self.held, self.new = cfg, np.array(held), np.array(new)
        self.ctx = self.held + self.new
        B = len(held)
        pps = int(max(1, (self.ctx.max() + PAGE - 1) // PAGE)) + 1
        self.n_pages = int(sum(-(-c // PAGE) for c in self.ctx)) + spare
        self.table = torch.full((B, pps), -1, dtype=torch.int32, device="cuda")
        self.signs, self.S = signs_and_sketch(seed, cfg)
        self.cache = kvq.KvqCache(cfg, B, 0, self.signs, self.S, block_table=self.table, n_pages=self.n_pages)
        self.cache.arena[int(self.cache.layout()[4]):].fill_(0xFF)  # norms behind the tokens are NaN
        free = cuda_ints(rng.permutation(self.n_pages))
        cursor = cuda_ints([0])
        gen = torch.Generator(device="cuda").manual_seed(seed)
        zero = np.zeros(B, dtype=int)
        for have, take, last in ((zero, self.held, False), (self.held, self.new, True)):
            n = int(take.sum())
            self.seq_start, self.ctx_lens, taken = cuda_ints(np.zeros(B + 1)), cuda_ints(zero), cuda_ints([0, 0])
            kvq.kvq_extend_block_table(cuda_ints(have), cuda_ints(take), free, self.table, self.seq_start, self.ctx_lens,
                                       taken, cursor)
            cursor += taken[:1]
            seq, pos, slots = cuda_ints(np.zeros(n)), cuda_ints(np.zeros(n)), cuda_ints(np.zeros(n), torch.int64)
            kvq.kvq_slot_map(cuda_ints(have), self.seq_start, self.ctx_lens, self.table, self.n_pages, seq, pos, slots)
            kv = [torch.randn(n, cfg.n_kv_heads, 128, generator=gen, device="cuda").to(dtype) for _ in range(2)]
            if last:
                kv = [kv[0] if k is None else k, kv[1] if v is None else v]
            self.cache.quantize_slots(*kv, slots)
        self.q = (1.5 * torch.randn(int(self.new.sum()), cfg.n_q_heads, 128, generator=gen, device="cuda")).to(dtype)

    def reference(self, q=None):
        q = (self.q if q is None else q).double().cpu().numpy()
        out, table, g = np.zeros(q.shape), self.table.cpu().numpy(), self.cfg.n_q_heads // self.cfg.n_kv_heads
        start = np.concatenate([[0], np.cumsum(self.new)])
        for b, T in enumerate(self.ctx):
            rows = slice(start[b], start[b + 1])
            for hk in range(self.cfg.n_kv_heads):
                K, V = dequantised(self.cache, self.cfg, table, b, hk, int(T), self.signs, self.S)
                out[rows, hk * g:(hk + 1) * g] = causal_attention(q[rows, hk * g:(hk + 1) * g], K, V, int(T))
        return out


def assert_close(out, ref, dtype):
    """fp32: 1e-4 of a row's largest entry: the logits' fp32 sums of 256 products stay within 256 * 2^-24 of
    sum |q k| < 100, so weights are off by less than 2e-3 at the very worst and a hundredth of that in
    earnest (errors of either sign). bf16: operands rounded to fp16, queries and keys 2^-11 each of an
    entry, keys twice (code and norm): a logit is off by about sqrt(3) 2^-11 |q k|_2 < 1.3e-3 (one sigma;
    |q k|_2 about 1.5), a row's weighted mean of independent vectors by as much of its own size; four sigma
    is 5e-3 of the largest entry, the weights' and values' own roundings included; then the output's half
    step, 2^-8 of an entry."""
    out, ref = out.double().cpu().numpy(), np.asarray(ref)
    top = np.abs(ref).max(-1, keepdims=True)
    tol = 1e-4 * top if dtype == torch.float32 else 5e-3 * top + 2.0 ** -8 * np.abs(ref)
    worst = np.abs(out - ref) / np.maximum(tol, 1e-30)
    assert np.isfinite(out).all() and worst.max() <= 1, f"{worst.max():.3f} of the tolerance"
