"""Measured cases of the ragged serving path over a paged few-bit cache, and the operators' plain forms.

A serving step that mixes prompts and single tokens runs four operators in a row:

  extend_block_table  pages for the new tokens of every request, from request lengths, on the GPU
  slot_map            request, position and page slot of every new token
  quantize_slots      code the new keys and values and write them into their slots
  chunk_attention     attention of the new tokens over the packed pages, causal in each request

Cases are dicts of plain values; `lens` seeds the ragged lengths, so that the work of a case does not
depend on the seed of its data.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128          # head dimension
PAGE = 64        # tokens of a page: two tiles of 32
TILE = 32
INT32 = torch.int32


# ---- cases ------------------------------------------------------------------------------------------


def _table_case(name, batch, held_lo, held_hi, new_lo, new_hi, lens, op):
    return {"name": name, "op": op, "batch": batch, "held_lo": held_lo, "held_hi": held_hi, "new_lo": new_lo,
            "new_hi": new_hi, "lens": lens}


def _cache_case(name, op, batch, hq, hkv, kb, kq, vb, vq, held_lo, held_hi, new_lo, new_hi, dtype, lens):
    return {"name": name, "op": op, "batch": batch, "hq": hq, "hkv": hkv, "k_bits": kb, "k_qjl": kq, "v_bits": vb,
            "v_qjl": vq, "held_lo": held_lo, "held_hi": held_hi, "new_lo": new_lo, "new_hi": new_hi, "dtype": dtype,
            "lens": lens}


def listed():
    return [
        # a decode step of 16 requests: one token each, a page now and then
        _table_case("table_decode16", 16, 1, 8192, 1, 1, 1, "extend_block_table"),
        # admission of 256 prompts beside running requests
        _table_case("table_admit256", 256, 0, 16384, 1, 16000, 2, "extend_block_table"),
        # the slots of one decode step
        _table_case("slots_decode16", 16, 1, 8192, 1, 1, 3, "slot_map"),
        # the slots of a large mixed batch of prompts
        _table_case("slots_prompts64", 64, 0, 8192, 1, 4000, 4, "slot_map"),
        # an 8B-shaped decode step with a few speculated tokens per request
        _cache_case("append_verify_8b", "quantize_slots", 16, 32, 8, 2, True, 2, True, 1, 500, 1, 8, "bf16", 5),
        # a 70B-shaped prefill chunk of ragged prompts
        _cache_case("append_chunk_70b", "quantize_slots", 4, 64, 8, 3, True, 3, False, 0, 300, 400, 700, "bf16", 6),
        # fp32 keys and values, one sign bit per coordinate
        _cache_case("append_sign_f32", "quantize_slots", 3, 8, 2, 1, False, 1, False, 0, 200, 1, 301, "f32", 7),
        # an 8B-shaped verification step: up to 8 speculated tokens per request over a long cache
        _cache_case("chunk_verify_8b", "chunk_attention", 16, 32, 8, 2, True, 2, True, 6000, 8184, 1, 8, "bf16", 8),
        # a 70B-shaped prefill chunk of one long prompt
        _cache_case("chunk_prefill_70b", "chunk_attention", 1, 64, 8, 3, True, 3, False, 30720, 30720, 2048, 2048, "bf16",
                    9),
        # prompt chunks and single tokens of an 8B-shaped layer in one batch
        _cache_case("chunk_mixed_8b", "chunk_attention", 8, 32, 8, 2, True, 2, True, 0, 4000, 1, 513, "bf16", 10),
        # one sign bit per coordinate, medium chunks over 16384 tokens
        _cache_case("chunk_onebit", "chunk_attention", 4, 32, 8, 1, False, 1, False, 12000, 16000, 100, 384, "bf16", 11),
        # the smallest: a few fp32 tokens of one head
        _cache_case("chunk_tiny_f32", "chunk_attention", 1, 1, 1, 2, True, 2, True, 1000, 1000, 7, 7, "f32", 12),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["extend_block_table", "slot_map", "quantize_slots", "chunk_attention", "chunk_attention"])
    lens = rng.randrange(1 << 30)
    if op in ("extend_block_table", "slot_map"):
        batch = _log_int(rng, 1, 256)
        held = _log_int(rng, 1, 16384)
        new = _log_int(rng, 1, 16000 if op == "extend_block_table" else max(1, 200000 // batch))
        case = _table_case("", batch, 0, held, 1, min(new, 16000), lens, op)
    else:
        kb, kq, vb, vq = rng.choice([(2, True, 2, True), (3, True, 3, False), (1, False, 1, False), (2, True, 2, False),
                                     (3, True, 3, True), (2, False, 2, False), (3, False, 3, False)])
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 4, 8])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        batch = _log_int(rng, 1, 16)
        if op == "quantize_slots":
            new = _log_int(rng, 1, max(1, 2048 // batch))
            case = _cache_case("", op, batch, hq, hkv, kb, kq, vb, vq, 0, _log_int(rng, 1, 500), 1, new, dtype, lens)
        else:
            new = _log_int(rng, 1, max(1, 2048 // batch if dtype == "bf16" else 256 // batch))
            held = _log_int(rng, 1, 32000 // batch)
            case = _cache_case("", op, batch, hq, hkv, kb, kq, vb, vq, held // 2, held, max(1, new // 4), new, dtype, lens)
    del case["name"]
    return case


def _lengths(case):
    """(tokens held, new tokens) of every request of a case, ragged by its `lens`."""
    rng = random.Random(case["lens"])
    held = [rng.randint(case["held_lo"], case["held_hi"]) for _ in range(case["batch"])]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(case["batch"])]
    return held, new


def _pages(tokens):
    return -(-tokens // PAGE)


# ---- the codec's tables and the packed layout -------------------------------------------------------


def _lloyd_max(bits):
    """Centroids and thresholds (fp32 values) of the Gaussian Lloyd-Max quantizer: the fixed point of cell means."""
    n = 1 << bits
    c = np.linspace(-1.5, 1.5, n) if n > 1 else np.zeros(1)
    phi = lambda x: np.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)  # noqa: E731
    cdf = lambda x: 0.5 * np.array([math.erfc(-v / math.sqrt(2)) for v in x])  # noqa: E731
    for _ in range(4000):
        t = 0.5 * (c[1:] + c[:-1])
        edge = np.concatenate([[-40.0], t, [40.0]])
        c = -(phi(edge[1:]) - phi(edge[:-1])) / (cdf(edge[1:]) - cdf(edge[:-1]))
        c = 0.5 * (c - c[::-1])
    c32 = c.astype(np.float32)
    return c32, (0.5 * (c[1:] + c[:-1])).astype(np.float32)


TABLES = {bits: _lloyd_max(bits) for bits in (1, 2, 3)}


def _hadamard(dtype, device):
    h = torch.ones(1, 1, dtype=dtype, device=device)
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _tile_bytes(bits, qjl):
    return bits * 512 + (512 if qjl else 0) + 64 + (64 if qjl else 0)


def _pack(bits, octet):
    """0/1 bits uint8 [..., 32 tokens, planes, 128] -> bytes [..., planes * 512] in a tile's order."""
    lead, planes = bits.shape[:-3], bits.shape[-2]
    shift = torch.arange(8, dtype=torch.uint8, device=bits.device)
    b = bits.transpose(-3, -2)  # [..., planes, 32, 128]
    if octet:  # byte (octet, t, m, h, i): coordinate 32 m + 16 h + 4 t + i, bit j is token 8 octet + j
        b = b.reshape(*lead, planes, 4, 8, 4, 2, 4, 4)  # [o, j, m, h, t, i]
        n = len(lead) + 1
        b = b.permute(*range(n), n, n + 4, n + 2, n + 3, n + 5, n + 1)
        out = (b << shift).sum(-1, dtype=torch.uint8)
    else:      # byte (lane k, token): bit i is coordinate 8 k + i
        b = b.reshape(*lead, planes, 32, 16, 8)
        out = (b << shift).sum(-1, dtype=torch.uint8).transpose(-1, -2)
    return out.reshape(*lead, planes * 512)


def _unpack(raw, planes, octet):
    """The inverse of _pack."""
    lead = raw.shape[:-1]
    shift = torch.arange(8, dtype=torch.uint8, device=raw.device)
    if octet:
        b = (raw.reshape(*lead, planes, 4, 4, 4, 2, 4, 1) >> shift) & 1  # [o, t, m, h, i, j]
        n = len(lead) + 1
        b = b.permute(*range(n), n, n + 5, n + 2, n + 3, n + 1, n + 4)
    else:
        b = (raw.reshape(*lead, planes, 16, 32, 1).transpose(-2, -3) >> shift) & 1
    return b.reshape(*lead, planes, 32, 128).transpose(-3, -2)


def _tiles(codes, z, norm, gamma, bits, octet):
    """Bytes [..., tile_bytes] of tiles: codes uint8 [..., 32, 128], z the same or None, norm and gamma fp16 [..., 32]."""
    shift = torch.arange(bits, dtype=torch.uint8, device=codes.device)[:, None]
    planes = (codes[..., None, :] >> shift) & 1
    if z is not None:
        planes = torch.cat([planes, z[..., None, :]], -2)
    parts = [_pack(planes, octet), norm.contiguous().view(torch.uint8)]
    if z is not None:
        parts.append(gamma.contiguous().view(torch.uint8))
    return torch.cat(parts, -1)


def _fields(tiles, bits, qjl, octet):
    """The inverse of _tiles."""
    n = bits + (1 if qjl else 0)
    planes = _unpack(tiles[..., :n * 512], n, octet)
    shift = torch.arange(bits, dtype=torch.uint8, device=tiles.device)[:, None]
    codes = (planes[..., :bits, :] << shift).sum(-2, dtype=torch.uint8)
    tail = tiles[..., n * 512:].contiguous().view(torch.float16)
    return codes, planes[..., bits, :] if qjl else None, tail[..., :32], tail[..., 32:] if qjl else None


# ---- inputs -----------------------------------------------------------------------------------------


def _random_pool(gen, n_pages, hkv, bits, qjl, octet, S, spread):
    """Packed pages [n_pages, hkv, 2, tile_bytes] of Gaussian coordinates (rotated keys and values are close to
    that), with norms spread as exp(spread * normal) around sqrt(128)."""
    cent, thr = (torch.tensor(x, device="cuda") for x in TABLES[bits])
    pool = torch.empty(n_pages, hkv, 2, _tile_bytes(bits, qjl), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 18) // (hkv * PAGE))
    for first in range(0, n_pages, step):
        part = pool[first:first + step]
        u = torch.randn(*part.shape[:3], TILE, D, generator=gen, device="cuda")
        codes = torch.bucketize(u, thr, right=True)
        norm = (math.sqrt(D) * torch.exp(spread * torch.randn(u.shape[:-1], generator=gen, device="cuda"))).half()
        z = gamma = None
        if qjl:
            rho = u - cent[codes]
            gamma = rho.norm(dim=-1).half()
            z = (rho @ S.T >= 0).to(torch.uint8)
        part.copy_(_tiles(codes.to(torch.uint8), z, norm, gamma, bits, octet))
    return pool


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed & 0x7FFFFFFFFFFFFFFF)


def _rotated(x, signs):
    """Norms and rotated, normalised vectors in 64 bits (a zero vector gives zeros)."""
    x = x.double()
    n = (x * x).sum(-1).sqrt()
    y = (x * signs.double()) @ _hadamard(torch.float64, x.device)
    return n, torch.where(n[..., None] > 0, y / n[..., None], torch.zeros((), dtype=torch.float64, device=x.device))


def _decided(x, signs, S, bits, qjl):
    """x with every vector that lies within rounding of a code, sign or fp16 border replaced by one that does not."""
    cent, thr = (torch.tensor(v, device=x.device, dtype=torch.float64) for v in TABLES[bits])
    flat = x.reshape(-1, D)
    n, u = _rotated(flat, signs)
    def tie(v):  # distance from the nearest midpoint of two fp16 numbers, in ulps
        _, e = torch.frexp(v)
        w = v * torch.exp2(11.0 - e)
        return (w - w.floor() - 0.5).abs()
    good = ((u[..., None] - thr).abs().amin((-1, -2)) > 2e-5) & (tie(n) > 0.02)
    if qjl:
        rho = u - cent[(u[..., None] >= thr).sum(-1)]
        good &= ((rho @ S.double().T).abs().amin(-1) > 2e-4) & (tie((rho * rho).sum(-1).sqrt()) > 0.02)
    keep = torch.nonzero(good)[:, 0]
    pick = torch.where(good, torch.arange(len(flat), device=x.device), keep[torch.arange(len(flat), device=x.device) % len(keep)])
    return flat[pick].reshape(x.shape).contiguous()


def _cache(case, table, n_pages, k_pool, v_pool, signs, S):
    """The framework's paged cache of a case, holding the pools' bytes."""
    import bit_kv_cache_seeded_b200 as kvq

    mode = lambda bits, qjl: "lm_qjl" if qjl else ("sign1" if bits == 1 else "lm")  # noqa: E731
    cfg = kvq.make_cfg(D, case["hq"], case["hkv"], mode(case["k_bits"], case["k_qjl"]), mode(case["v_bits"], case["v_qjl"]),
                       case["k_bits"], case["v_bits"], D if case["k_qjl"] or case["v_qjl"] else 0)
    cache = kvq.KvqCache(cfg, case["batch"], 0, signs.cpu().numpy(), None if S is None else S.cpu().numpy(),
                         block_table=table, n_pages=n_pages)
    info = cache.layout()
    views = []
    for off, pool in ((int(info[4]), k_pool), (int(info[5]), v_pool)):
        region = cache.arena[off:off + pool.numel()].view(pool.shape)
        region.copy_(pool)
        views.append(region)
    return cache, views


def prepare(case, seed):
    gen = _generator(seed)
    held, new = _lengths(case)
    op, batch = case["op"], case["batch"]
    dev = lambda v: torch.tensor(v, dtype=INT32, device="cuda")  # noqa: E731
    after = [h + n for h, n in zip(held, new)]
    pps = _pages(max(after)) + 1
    n_pages = sum(_pages(a) for a in after) + 5
    perm = torch.randperm(n_pages, generator=gen, device="cuda").to(INT32)
    state = {"op": op, "held": dev(held), "new": dev(new), "n_pages": n_pages}
    if op == "extend_block_table":
        # pages that the requests hold already come first in the shuffled pool, the free ones after them
        table = torch.full((batch, pps), -1, dtype=INT32, device="cuda")
        counts = torch.tensor([_pages(h) for h in held], device="cuda")
        taken = torch.arange(pps, device="cuda") < counts[:, None]
        table[taken] = perm[:int(counts.sum())]
        state |= {"table": table, "free": perm[int(counts.sum()):].contiguous(),
                  "seq_start": torch.empty(batch + 1, dtype=INT32, device="cuda"),
                  "ctx_lens": torch.empty(batch, dtype=INT32, device="cuda"),
                  "taken": torch.empty(2, dtype=INT32, device="cuda")}
        return state
    counts = torch.tensor([_pages(a) for a in after], device="cuda")
    table = torch.full((batch, pps), -1, dtype=INT32, device="cuda")
    table[torch.arange(pps, device="cuda") < counts[:, None]] = perm[:int(counts.sum())]
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=INT32, device="cuda")
    n_tokens = sum(new)
    state |= {"table": table, "seq_start": start, "ctx_lens": dev(after)}
    if op == "slot_map":
        state |= {"seq_ids": torch.empty(n_tokens, dtype=INT32, device="cuda"),
                  "positions": torch.empty(n_tokens, dtype=INT32, device="cuda"),
                  "slots": torch.empty(n_tokens, dtype=torch.int64, device="cuda")}
        return state
    state["case"] = case
    signs = (torch.randint(0, 2, (D,), generator=gen, device="cuda") * 2 - 1).to(torch.int8)
    S = torch.randn(D, D, generator=gen, device="cuda") if case["k_qjl"] or case["v_qjl"] else None
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    k_pool = _random_pool(gen, n_pages, case["hkv"], case["k_bits"], case["k_qjl"], True, S, 0.25)
    v_pool = _random_pool(gen, n_pages, case["hkv"], case["v_bits"], case["v_qjl"], False, S, 0.25)
    state |= {"signs": signs, "S": S}
    if own:
        state["cache"], (k_pool, v_pool) = _cache(case, table, n_pages, k_pool, v_pool, signs, S)
    state |= {"k_pool": k_pool, "v_pool": v_pool}
    if op == "quantize_slots":
        # keys carry a few outlier channels, as trained models' keys do
        k = torch.randn(n_tokens, case["hkv"], D, generator=gen, device="cuda")
        k[..., ::21] *= 15.0
        v = torch.randn(n_tokens, case["hkv"], D, generator=gen, device="cuda")
        state["k"] = _decided(k.to(dtype), signs, S, case["k_bits"], case["k_qjl"])
        state["v"] = _decided(v.to(dtype), signs, S, case["v_bits"], case["v_qjl"])
        t = torch.arange(n_tokens, device="cuda")
        seq = torch.searchsorted(start[1:].long(), t, right=True)
        pos = state["held"].long()[seq] + t - start.long()[seq]
        state["slots"] = table.long()[seq, pos // PAGE] * PAGE + pos % PAGE
        return state
    state["q"] = (1.5 * torch.randn(n_tokens, case["hq"], D, generator=gen, device="cuda")).to(dtype)
    return state


# ---- one pass ---------------------------------------------------------------------------------------


def _plain_extend_block_table(s):
    held, new, table, free = s["held"].long(), s["new"].long(), s["table"], s["free"]
    pps = table.shape[1]
    ok = (held >= 0) & (new >= 0) & (held + new <= pps * PAGE)
    p0, p1 = (held + PAGE - 1) // PAGE, (held + new + PAGE - 1) // PAGE
    need = torch.where(ok, p1 - p0, 0)
    end = torch.cumsum(need, 0)
    ok &= (need == 0) | (end <= free.numel())
    page = torch.arange(pps, device=table.device)
    write = ok[:, None] & (page >= p0[:, None]) & (page < p1[:, None])
    source = torch.where(write, (end - need - p0)[:, None] + page, 0)
    out = torch.where(write, free[source.clamp(max=free.numel() - 1)], table)
    start = torch.cat([torch.zeros(1, dtype=torch.int64, device=table.device), torch.cumsum(new.clamp(min=0), 0)])
    ctx = torch.where(ok, held + new, held.clamp(0, pps * PAGE))
    taken = torch.stack([(need * ok).sum(), (~ok).sum()])
    return out, start.to(INT32), ctx.to(INT32), taken.to(INT32)


def _plain_slot_map(s):
    start, held, table = s["seq_start"].long(), s["held"].long(), s["table"].long()
    t = torch.arange(s["slots"].numel(), device=table.device)
    seq = torch.searchsorted(start[1:], t, right=True)
    pos = held[seq] + t - start[seq]
    page = table[seq, pos // PAGE]
    granted = s["ctx_lens"].long()[seq] == held[seq] + start[seq + 1] - start[seq]
    good = granted & (page >= 0) & (page < s["n_pages"])
    return seq.to(INT32), pos.to(INT32), torch.where(good, page * PAGE + pos % PAGE, -1)


def _plain_append(pool, x, slots, signs, S, bits, qjl, octet):
    cent, thr = (torch.tensor(v, device=x.device, dtype=torch.float64) for v in TABLES[bits])
    n, u = _rotated(x, signs)  # 64 bits: a value next to a threshold decides a code
    code = (u[..., None] >= thr).sum(-1)
    codes, z, norm, gamma = _fields(pool, bits, qjl, octet)
    page, tile, tok = slots // PAGE, slots % PAGE // TILE, slots % TILE
    codes = codes.clone()
    codes[page, :, tile, tok] = code.to(torch.uint8)
    norm = norm.clone()
    norm[page, :, tile, tok] = n.half()
    if qjl:
        rho = u - cent[code]
        gamma, z = gamma.clone(), z.clone()
        gamma[page, :, tile, tok] = (rho * rho).sum(-1).sqrt().half()
        z[page, :, tile, tok] = (rho @ S.double().T >= 0).to(torch.uint8)
    return _tiles(codes, z, norm, gamma, bits, octet)


def _plain_dequantised(pool, table, S, bits, qjl, octet):
    """Rotated keys or values fp32 [batch, hkv, pages * 64, 128] of the pages that a block table names."""
    tiles = pool[table.long().clamp(min=0)]  # [batch, pages, hkv, 2, bytes]
    codes, z, norm, gamma = _fields(tiles, bits, qjl, octet)
    cent = torch.tensor(TABLES[bits][0], device=pool.device)
    x = cent[codes.int()]
    if qjl:
        x += math.sqrt(math.pi / 2) / D * gamma.float()[..., None] * ((2.0 * z.float() - 1) @ S)
    x *= norm.float()[..., None] / math.sqrt(D)
    b, p, h = x.shape[:3]
    return x.permute(0, 2, 1, 3, 4, 5).reshape(b, h, p * PAGE, D)


def _plain_chunk_attention(s):
    c, q, start, ctx = s["case"], s["q"], s["seq_start"].long(), s["ctx_lens"].long()
    k = _plain_dequantised(s["k_pool"], s["table"], s["S"], c["k_bits"], c["k_qjl"], True)
    v = _plain_dequantised(s["v_pool"], s["table"], s["S"], c["v_bits"], c["v_qjl"], False)
    H, group = _hadamard(torch.float32, q.device), c["hq"] // c["hkv"]
    rotated = (q.float() * s["signs"].float()) @ H / math.sqrt(D)
    # rows of the requests side by side, padded to the longest chunk
    t = torch.arange(q.shape[0], device=q.device)
    seq = torch.searchsorted(start[1:], t, right=True)
    row = t - start[seq]
    longest = c["new_hi"]
    padded = torch.zeros(c["batch"], longest, c["hq"], D, device=q.device)
    padded[seq, row] = rotated
    padded = padded.reshape(c["batch"], longest, c["hkv"], group, D).permute(0, 2, 3, 1, 4)
    logits = (padded.reshape(c["batch"], c["hkv"], group * longest, D) @ k.transpose(-1, -2)) / math.sqrt(D)
    logits = logits.reshape(c["batch"], c["hkv"], group, longest, -1)
    limit = (ctx - (start[1:] - start[:-1]))[:, None] + torch.arange(longest, device=q.device)  # own position
    masked = torch.arange(logits.shape[-1], device=q.device) > limit.clamp(max=(ctx - 1)[:, None])[..., None]
    logits.masked_fill_(masked[:, None, None], -math.inf)
    top = logits.amax(-1, keepdim=True)
    logits.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = logits.sum(-1, keepdim=True)
    out = logits.reshape(c["batch"], c["hkv"], group * longest, -1) @ v
    out = out.reshape(c["batch"], c["hkv"], group, longest, D) / torch.where(total > 0, total, 1.0)
    out = out.permute(0, 3, 1, 2, 4).reshape(c["batch"], longest, c["hq"], D)[seq, row]
    return ((out @ H) * s["signs"].float() / math.sqrt(D)).to(q.dtype)


def run(state):
    s = state
    if s["op"] == "extend_block_table":
        if own:
            import bit_kv_cache_seeded_b200 as kvq

            kvq.kvq_extend_block_table(s["held"], s["new"], s["free"], s["table"], s["seq_start"], s["ctx_lens"], s["taken"])
            return s["table"], s["seq_start"], s["ctx_lens"], s["taken"]
        return _plain_extend_block_table(s)
    if s["op"] == "slot_map":
        if own:
            import bit_kv_cache_seeded_b200 as kvq

            kvq.kvq_slot_map(s["held"], s["seq_start"], s["ctx_lens"], s["table"], s["n_pages"], s["seq_ids"], s["positions"],
                             s["slots"])
            return s["seq_ids"], s["positions"], s["slots"]
        return _plain_slot_map(s)
    if s["op"] == "quantize_slots":
        if own:
            s["cache"].quantize_slots(s["k"], s["v"], s["slots"])
            return s["k_pool"], s["v_pool"]
        c = s["case"]
        return (_plain_append(s["k_pool"], s["k"], s["slots"], s["signs"], s["S"], c["k_bits"], c["k_qjl"], True),
                _plain_append(s["v_pool"], s["v"], s["slots"], s["signs"], s["S"], c["v_bits"], c["v_qjl"], False))
    if own:
        return s["cache"].chunk_attention(s["q"], s["seq_start"], s["ctx_lens"])
    return _plain_chunk_attention(s)


# ---- the work of a case, and its result in 64 bits --------------------------------------------------


def work(case):
    held, new = _lengths(case)
    op, batch, tokens = case["op"], case["batch"], sum(new)
    pages = sum(_pages(h + n) - _pages(h) for h, n in zip(held, new))
    if op == "extend_block_table":  # lengths in; offsets, lengths and the new pages' entries out
        return {"bytes": 4 * (2 * batch + 2 * batch + 1 + 2 + 2 * pages), "flops": 0}
    if op == "slot_map":            # request, position and slot of every token; offsets, lengths and entries in
        return {"bytes": 16 * tokens + 4 * (3 * batch + 1 + sum(_pages(n) for n in new)), "flops": 0}
    elem = 2 if case["dtype"] == "bf16" else 4
    side = [_tile_bytes(case["k_bits"], case["k_qjl"]) / TILE, _tile_bytes(case["v_bits"], case["v_qjl"]) / TILE]
    if op == "quantize_slots":      # keys and values in, packed bytes out; rotation, and the sketch's products
        flops = sum((2 * D * D if qjl else 0) + 7 * D for qjl in (case["k_qjl"], case["v_qjl"])) * tokens * case["hkv"]
        return {"bytes": tokens * (8 + case["hkv"] * (2 * D * elem + sum(side))), "flops": flops}
    ctx = sum(h + n for h, n in zip(held, new))
    pairs = sum(n * h + n * (n + 1) // 2 for h, n in zip(held, new)) * case["hq"]
    # the packed cache once, queries in, outputs out; two products over the attended pairs
    return {"bytes": ctx * case["hkv"] * sum(side) + 2 * tokens * case["hq"] * D * elem, "flops": 4 * D * pairs}


def exact(case, seed):
    if case["op"] != "chunk_attention":
        return None  # whole numbers
    s = prepare(case, seed)
    held, new = _lengths(case)
    signs = s["signs"].double()
    H = _hadamard(torch.float64, signs.device)
    sides = []
    for pool, bits, qjl, octet in ((s["k_pool"], case["k_bits"], case["k_qjl"], True),
                                   (s["v_pool"], case["v_bits"], case["v_qjl"], False)):
        sides.append((pool, bits, qjl, octet, torch.tensor(TABLES[bits][0], device=pool.device).double()))
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    group, first = case["hq"] // case["hkv"], 0
    for b, (h, n) in enumerate(zip(held, new)):
        pages = s["table"][b, :_pages(h + n)].long()
        reach = torch.arange(h + n, device=out.device) <= (h + torch.arange(n, device=out.device))[:, None]
        for head in range(case["hkv"]):
            kv = []
            for pool, bits, qjl, octet, cent in sides:
                codes, z, norm, gamma = (None if f is None else f.flatten(0, 3) for f in
                                         _fields(pool[pages][:, head:head + 1], bits, qjl, octet))
                est = cent[codes.long()]
                if qjl:
                    est = est + math.sqrt(math.pi / 2) / D * gamma.double()[:, None] * ((2 * z.double() - 1) @ s["S"].double())
                x = est * norm.double()[:, None] / math.sqrt(D)
                kv.append(((x @ H) * signs / math.sqrt(D))[:h + n])  # back in the unrotated domain
            for g in range(head * group, (head + 1) * group):
                logits = s["q"][first:first + n, g].double() @ kv[0].T / math.sqrt(D)
                out[first:first + n, g] = torch.softmax(logits.masked_fill(~reach, -math.inf), -1) @ kv[1]
        first += n
    return out
