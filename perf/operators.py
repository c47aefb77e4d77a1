"""The 4-bit KV cache operators: what a step over such a cache runs, in a plain form and through the package.

Four operators make one decode or mixed step whose cache is held in 4 bits:

* tables -- the step's row offsets, positions, slots and block table, built on the GPU from the requests'
  lengths, with new pages taken from a free list;
* append -- the rotary embedding at absolute positions, and the paged append of K and V in 4 bits;
* read   -- cached rows by slot, as the bf16 values that they stand for;
* attend -- causal attention of every packed row over its pages of the 4-bit cache.

The 4-bit form.  A cached row of one token and KV head is cut into groups of 32 consecutive elements.  A group
holds s = r5(max|x| / 7) and the codes rint(x / s) in -7..7, with r5 the rounding to five significant bits
(nearest, ties to even); it stands for s * code, which bf16 holds exactly.  A page of one KV head is one block
of 16 D + 2 D bytes: the codes of 16 K rows, those of 16 V rows (code + 8 in a nibble, ordered as `pack` below
lays them out), the 16 x D/32 scales of K and those of V (bf16).
"""
import math
import random

import torch

own = False

PAGE = 16
GROUP = 32


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the metadata of a decode-only step: 64 requests of a 32-head layer, one new token each
        {"name": "tables_decode_64", "op": "tables", "decodes": 64, "ctx_lo": 512, "ctx_hi": 4096, "chunks": 0,
         "chunk_tokens": 0, "chunk_start": 0, "chunk_step": 0, "ragged": False},
        # a long bimodal step: 512 decodes up to 128K keys next to the last 4096 tokens of a 32K prompt
        {"name": "tables_mixed_512", "op": "tables", "decodes": 512, "ctx_lo": 200, "ctx_hi": 131072, "chunks": 1,
         "chunk_tokens": 4096, "chunk_start": 28672, "chunk_step": 0, "ragged": True},
        # the append of a decode-only step: one token for each of 64 requests, 32 KV heads
        {"name": "append_decode_64", "op": "append", "tokens": 64, "H_q": 32, "H_kv": 32, "D": 128, "ctx_hi": 4096},
        # the append of a full mixed step with grouped heads: 8192 tokens, most of them prompt chunks
        {"name": "append_mixed_8192", "op": "append", "tokens": 8192, "H_q": 32, "H_kv": 8, "D": 128, "ctx_hi": 16384},
        # one request's last rows read back, a small odd number of them
        {"name": "read_rows_37", "op": "read", "tokens": 37, "H_kv": 2, "D": 64},
        # a cached prefix of 6000 tokens handed to a bf16 cache
        {"name": "read_prefix_6000", "op": "read", "tokens": 6000, "H_kv": 8, "D": 128},
        # the smallest step: three short decodes and a 5-token chunk, where the latency of a call counts
        {"name": "attend_small_8", "op": "attend", "H_q": 4, "H_kv": 2, "D": 64, "decodes": 3, "ctx_lo": 37,
         "ctx_hi": 100, "chunks": 1, "chunk_tokens": 5, "chunk_start": 0, "chunk_step": 0, "ragged": False},
        # decodes of a layer without shared heads: 64 requests, 512 to 4096 keys
        {"name": "attend_decode_mha_64", "op": "attend", "H_q": 32, "H_kv": 32, "D": 128, "decodes": 64,
         "ctx_lo": 512, "ctx_hi": 4096, "chunks": 0, "chunk_tokens": 0, "chunk_start": 0, "chunk_step": 0,
         "ragged": False},
        # decodes of a grouped-query layer: 256 requests, 700 to 16K keys
        {"name": "attend_decode_gqa_256", "op": "attend", "H_q": 32, "H_kv": 8, "D": 128, "decodes": 256,
         "ctx_lo": 700, "ctx_hi": 16384, "chunks": 0, "chunk_tokens": 0, "chunk_start": 0, "chunk_step": 0,
         "ragged": True},
        # prompt chunks alone: a whole 3968-token prompt and a chunk of the same length at 6000
        {"name": "attend_chunk_gqa_2", "op": "attend", "H_q": 32, "H_kv": 8, "D": 128, "decodes": 0, "ctx_lo": 1,
         "ctx_hi": 1, "chunks": 2, "chunk_tokens": 3968, "chunk_start": 0, "chunk_step": 6000, "ragged": False},
        # odd sizes and eight query heads to a KV head, half the head dim: 777-token chunks next to 61 decodes
        {"name": "attend_odd_d64", "op": "attend", "H_q": 16, "H_kv": 2, "D": 64, "decodes": 61, "ctx_lo": 1,
         "ctx_hi": 5003, "chunks": 3, "chunk_tokens": 777, "chunk_start": 11, "chunk_step": 1501, "ragged": True},
        # the largest: long decodes (64K to 128K keys) next to the last chunk of a 32K prompt
        {"name": "attend_mixed_long", "op": "attend", "H_q": 32, "H_kv": 8, "D": 128, "decodes": 16, "ctx_lo": 65536,
         "ctx_hi": 131072, "chunks": 1, "chunk_tokens": 4096, "chunk_start": 28672, "chunk_step": 0, "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "read", "attend", "attend", "attend"])
    G = rng.choice([1, 2, 4, 8])
    H_kv = rng.choice([1, 2, 4, 8, 10] if G > 2 else [2, 8, 16, 32, 40])
    H_q, D = G * H_kv, rng.choice([64, 128])
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 8192), "H_q": H_q, "H_kv": H_kv, "D": D, "ctx_hi": _log(rng, 64, 16384)}
    if op == "read":
        return {"op": op, "tokens": _log(rng, 1, 8192), "H_kv": H_kv, "D": D}
    rows = _log(rng, 1, 256 if op == "attend" else 1024)
    most = 2_000_000 // rows // (max(1, H_kv // 8) if op == "attend" else 1)
    hi = _log(rng, 16, min(131072, max(32, most)))
    lo = rng.randint(1, hi)
    chunks = rng.choice([0, 1, 1, 2, 3])
    d = _log(rng, 2, 4096 // max(1, chunks)) if chunks else 0
    start = rng.choice([0, _log(rng, 1, 28672)]) if chunks else 0
    c = {"op": op, "decodes": rows, "ctx_lo": lo, "ctx_hi": hi, "chunks": chunks, "chunk_tokens": d,
         "chunk_start": start, "chunk_step": rng.randint(0, 2000) if chunks else 0, "ragged": rng.random() < 0.5}
    return {**c, "H_q": H_q, "H_kv": H_kv, "D": D} if op == "attend" else c


def _rows(case):
    """(c, d) of every row: the decodes' cached lengths spaced evenly over their logarithm, then the chunks."""
    n, lo, hi = case["decodes"], case["ctx_lo"], case["ctx_hi"]
    dec = [(int(round(lo * (hi / lo) ** (i / max(1, n - 1)))), 1) for i in range(n)]
    return dec + [(case["chunk_start"] + i * case["chunk_step"], case["chunk_tokens"]) for i in range(case["chunks"])]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def work(case):
    if case["op"] == "tables":
        rows = _rows(case)
        R, T = len(rows), sum(d for _, d in rows)
        pages = sum(_pages(c + d) for c, d in rows)
        new = sum(_pages(c + d) - _pages(c) for c, d in rows)
        table = pages if case["ragged"] else R * max(_pages(c + d) for c, d in rows)
        # lengths in, the pages in use read once; offsets, starts, contexts, positions, slots, the table out
        return {"bytes": 4 * (2 * R + (pages - new) + 2 * new + 3 * R + 1 + 2 * T + table), "flops": 0}
    if case["op"] == "read":
        n, H_kv, D = case["tokens"], case["H_kv"], case["D"]
        return {"bytes": 4 * n + n * H_kv * (D + D // 8) + 4 * n * H_kv * D, "flops": 2 * n * H_kv * D}
    H_q, H_kv, D = case["H_q"], case["H_kv"], case["D"]
    if case["op"] == "append":
        # q, k, v in, q_rot out, K and V in 4 bits out; and the same rows read back in bf16
        T = case["tokens"]
        row = 4 * H_q * D + 4 * H_kv * D + 4 * D + 8
        return {"bytes": T * (row + 2 * H_kv * (D + D // 8) + 4 * H_kv * D), "flops": T * (H_q + 4 * H_kv) * D * 3}
    rows = _rows(case)
    T = sum(d for _, d in rows)
    kv = sum(c + d for c, d in rows)
    pages = sum(_pages(c + d) for c, d in rows)
    pairs = sum(d * c + d * (d + 1) // 2 for c, d in rows)
    return {"bytes": kv * H_kv * (D + D // 8) + 4 * T * H_q * D + 4 * (pages + 4 * len(rows)), "flops": 4 * D * H_q * pairs}


# ------------------------------------------------------------------------------------------------ inputs

def _scale5(a):
    """r5(a / 7) of the groups' largest magnitudes, as fp32."""
    u = (a / 7.0).view(torch.int32)
    u = (u + 0x3FFFF + ((u >> 19) & 1)) & ~0x7FFFF
    return u.view(torch.float32)


def quantize(x):
    """Rows [..., D] of fp32 values that bf16 holds -> codes [..., D] (fp32 whole numbers) and scales [..., D/32]."""
    g = x.unflatten(-1, (-1, GROUP))
    s = _scale5(g.abs().amax(-1))
    codes = torch.where(s[..., None] > 0, torch.round(g / s[..., None]), 0.0)
    return codes.flatten(-2), s


def pack(kc, ks, vc, vs):
    """Pages of codes [n, H, 16, D] and scales [n, H, 16, D/32] -> blocks [n, H, 18 D] of bytes."""
    n, H, _, D = kc.shape
    NG = D // GROUP
    e = [(c + 8).to(torch.uint8).view(n, H, PAGE, NG, 4, 4, 2) for c in (kc, vc)]  # group, quarter, i, parity
    k = e[0].permute(0, 1, 2, 4, 3, 6, 5).reshape(n, H, 8 * D, 2)                 # quarter, group, parity, i
    v = e[1].permute(0, 1, 2, 4, 6, 3, 5).reshape(n, H, 8 * D, 2)                 # quarter, parity, group, i
    sc = [s.to(torch.bfloat16).reshape(n, H, PAGE * NG).view(torch.uint8) for s in (ks, vs)]
    return torch.cat([k[..., 0] | (k[..., 1] << 4), v[..., 0] | (v[..., 1] << 4)] + sc, dim=-1)


def unpack(blocks, D):
    """Blocks [..., 18 D] -> K and V rows [..., 16, D] as fp32."""
    NG = D // GROUP
    lead = blocks.shape[:-1]
    nib = lambda b: torch.stack([b & 15, b >> 4], -1)  # noqa: E731
    n = len(lead)
    k = nib(blocks[..., : 8 * D]).reshape(*lead, PAGE, 4, NG, 2, 4).permute(*range(n + 1), n + 2, n + 1, n + 4, n + 3)
    v = nib(blocks[..., 8 * D: 16 * D]).reshape(*lead, PAGE, 4, 2, NG, 4).permute(*range(n + 1), n + 3, n + 1, n + 4, n + 2)
    sc = blocks[..., 16 * D:].contiguous().view(torch.bfloat16).reshape(*lead, 2, PAGE, NG, 1).float()
    k = (k.reshape(*lead, PAGE, NG, GROUP).float() - 8.0) * sc[..., 0, :, :, :]
    v = (v.reshape(*lead, PAGE, NG, GROUP).float() - 8.0) * sc[..., 1, :, :, :]
    return k.flatten(-2), v.flatten(-2)


def _pool(n, H, D, gen):
    """A pool of n pages whose rows are N(0, 1) values held in 4 bits."""
    pool = torch.empty((n, H, 18 * D), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (H * PAGE * D))
    for p in range(0, n, step):
        m = min(step, n - p)
        q = []
        for _ in range(2):
            x = torch.randn((m, H, PAGE, D), generator=gen, device="cuda").to(torch.bfloat16).float()
            q += list(quantize(x))
        pool[p: p + m] = pack(*q)
    return pool


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    if case["op"] == "append":
        T, H_q, H_kv, D = case["tokens"], case["H_q"], case["H_kv"], case["D"]
        pages = _pages(2 * T)
        slots = torch.randperm(PAGE * pages, generator=gen, device="cuda")[:T].to(torch.int32)
        pos = torch.randint(0, case["ctx_hi"], (T,), generator=gen, device="cuda", dtype=torch.int32)
        freq = 10000.0 ** (-torch.arange(0, D, 2, device="cuda", dtype=torch.float64) / D)
        ang = torch.arange(case["ctx_hi"], device="cuda", dtype=torch.float64)[:, None] * freq
        return {**case, "q": randn(T, H_q, D), "k": randn(T, H_kv, D), "v": randn(T, H_kv, D), "positions": pos,
                "slots": slots, "cos": ang.cos().float(), "sin": ang.sin().float(),
                "pool": torch.zeros((pages, H_kv, 18 * D), dtype=torch.uint8, device="cuda"),
                "q_rot": torch.empty((T, H_q, D), dtype=torch.bfloat16, device="cuda"),
                "k_out": torch.empty((T, H_kv, D), dtype=torch.bfloat16, device="cuda"),
                "v_out": torch.empty((T, H_kv, D), dtype=torch.bfloat16, device="cuda")}
    if case["op"] == "read":
        n, H_kv, D = case["tokens"], case["H_kv"], case["D"]
        pages = _pages(n) + 3
        order = torch.randperm(pages, generator=gen, device="cuda")  # a request's pages, rows in token order
        t = torch.arange(n, device="cuda")
        return {**case, "pool": _pool(pages, H_kv, D, gen), "slots": (order[t // PAGE] * PAGE + t % PAGE).to(torch.int32),
                "k_out": torch.empty((n, H_kv, D), dtype=torch.bfloat16, device="cuda"),
                "v_out": torch.empty((n, H_kv, D), dtype=torch.bfloat16, device="cuda")}
    rows = _rows(case)
    dec = rows[: case["decodes"]]
    r.shuffle(dec)
    rows = dec + rows[case["decodes"]:]
    need = [_pages(c + d) for c, d in rows]
    T, R, stride = sum(d for _, d in rows), len(rows), max(need)
    total = sum(need)
    if case["op"] == "tables":
        held = _ints([_pages(c) for c, _ in rows])
        new = total - int(held.sum())
        ids = torch.randperm(total + 100, generator=gen, device="cuda").to(torch.int32)
        j = torch.arange(stride, device="cuda")[None]
        first = (held.cumsum(0) - held)[:, None]
        table = torch.where(j < held[:, None], ids[(first + j).clamp(max=total - 1)], -1).to(torch.int32)
        cap = (T + 63) // 64 * 64  # tokens of the step's bucket
        out = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
        # the free pages, taken from the end: the ones that no table holds
        return {**case, "cached": _ints([c for c, _ in rows]), "new": _ints([d for _, d in rows]), "tables": table,
                "free": ids[total - new:].contiguous(), "free_count": _ints([new + 100]),
                "free_state": torch.zeros(2, dtype=torch.int32, device="cuda"), "pages": total + 100, "cap": cap,
                "used": total, "cu": out(R + 1), "start": out(R), "ctx": out(R), "positions": out(cap), "slots": out(cap),
                "bt": None if case["ragged"] else out(R, stride), "bt_offsets": out(R + 1) if case["ragged"] else None,
                "bt_pages": out(total) if case["ragged"] else None, "info": out(4)}
    H_q, H_kv, D = case["H_q"], case["H_kv"], case["D"]
    pool = _pool(total, H_kv, D, gen)
    ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    off = [0]
    for n in need:
        off.append(off[-1] + n)
    j = torch.arange(stride, device="cuda")[None]
    offs = _ints(off)
    bt = torch.where(j < _ints(need)[:, None], ids[(offs[:-1, None] + j).clamp(max=total - 1)], -1).to(torch.int32)
    cu = [0]
    for _, d in rows:
        cu.append(cu[-1] + d)
    return {**case, "q_rot": randn(T, H_q, D), "pool": pool, "cu": _ints(cu), "start": _ints([c for c, _ in rows]),
            "ctx": _ints([c + d for c, d in rows]), "bt": bt, "bt_offsets": offs, "bt_pages": ids,
            "context_total": sum(c + d for c, d in rows), "ctx_dec": max([c + 1 for c, _ in dec] or [0]),
            "ctx_chunk": max([c + d for c, d in rows[len(dec):]] or [0]),
            "out": torch.empty((T, H_q, D), dtype=torch.bfloat16, device="cuda")}


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_tables(st):
    c, d, free, count = st["cached"].long(), st["new"].long(), st["free"].long(), st["free_count"].long()
    R, cap = c.numel(), st["cap"]
    held, need = (c + 15) // PAGE, torch.where(d > 0, (c + d + 15) // PAGE, 0)
    new = (need - held).clamp(min=0)
    first = new.cumsum(0) - new
    j = torch.arange(st["tables"].shape[1], device=c.device)[None]
    fresh = (j >= held[:, None]) & (j < need[:, None])
    tables = torch.where(fresh, free[(count - 1 - first[:, None] - j + held[:, None]).clamp(0, free.numel() - 1)], st["tables"].long())
    cu = torch.cat([torch.zeros_like(c[:1]), d.cumsum(0)])
    t = torch.arange(cap, device=c.device)
    row = torch.searchsorted(cu[1:], t, right=True).clamp(max=R - 1)
    pos = torch.where(t < cu[-1], c[row] + t - cu[row], 0)
    slot = torch.where(t < cu[-1], tables[row, pos // PAGE] * PAGE + pos % PAGE, -1)
    out = {"cu": cu, "start": torch.where(d > 0, c, 0), "ctx": torch.where(d > 0, c + d, 0), "positions": pos, "slots": slot,
           "tables": tables, "free_count": count - new.sum(), "info": torch.stack([cu[-1], need.sum(), (d == 1).sum(), new.sum()])}
    if st["ragged"]:
        offs = torch.cat([torch.zeros_like(c[:1]), need.cumsum(0)])
        i = torch.arange(st["used"], device=c.device)
        row = torch.searchsorted(offs[1:], i, right=True)
        out |= {"bt_offsets": offs, "bt_pages": tables[row, i - offs[row]]}
    else:
        out["bt"] = torch.where(j < need[:, None], tables, -1)
    return {k: v.to(torch.int32) for k, v in out.items()}


def _plain_rotate(x, cos, sin):
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(torch.bfloat16)


def _plain_append(st):
    cos, sin = (st[n][st["positions"].long()][:, None] for n in ("cos", "sin"))
    q, k = _plain_rotate(st["q"], cos, sin), _plain_rotate(st["k"], cos, sin)
    held = [(c.unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2).to(torch.bfloat16)
            for c, s in (quantize(k.float()), quantize(st["v"].float()))]
    return {"q_rot": q, "k": held[0], "v": held[1]}


def _plain_read(st):
    D, slot = st["D"], st["slots"].long()
    k, v = unpack(st["pool"][slot // PAGE], D)  # [n, H, 16, D]
    at = (slot % PAGE)[:, None, None, None].expand(-1, st["H_kv"], 1, D)
    return {"k": k.gather(2, at).squeeze(2).to(torch.bfloat16), "v": v.gather(2, at).squeeze(2).to(torch.bfloat16)}


def _plain_rows(st, r0, r1, t0, d, keys):
    """Rows r0..r1-1, d tokens each from token t0 on, over at most `keys` keys."""
    H_q, H_kv, D, R, P = st["H_q"], st["H_kv"], st["D"], r1 - r0, _pages(keys)
    G = H_q // H_kv
    k, v = unpack(st["pool"][st["bt"][r0:r1, :P].long().clamp(min=0)], D)  # [R, P, H, 16, D]
    k, v = (x.transpose(1, 2).reshape(R, H_kv, P * PAGE, D) for x in (k, v))
    q = st["q_rot"][t0: t0 + R * d].float().view(R, d, H_kv, G, D).permute(0, 2, 3, 1, 4).reshape(R, H_kv, G * d, D)
    s = torch.matmul(q, k.transpose(-1, -2)).view(R, H_kv, G, d, P * PAGE) * (D ** -0.5)
    pos = st["start"][r0:r1].long()[:, None] + torch.arange(d, device=q.device)
    hidden = torch.arange(P * PAGE, device=q.device) > pos[:, None, None, :, None]
    s.masked_fill_(hidden, -math.inf)
    p = torch.exp(s - s.amax(-1, keepdim=True))
    o = torch.matmul(p.view(R, H_kv, G * d, P * PAGE), v).view(R, H_kv, G, d, D) / p.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(R * d, H_q, D).to(torch.bfloat16)


def _plain_attend(st):
    n, m = st["decodes"], st["chunks"]
    parts = [_plain_rows(st, 0, n, 0, 1, st["ctx_dec"])] if n else []
    if m:
        parts.append(_plain_rows(st, n, n + m, n, st["chunk_tokens"], st["ctx_chunk"]))
    return {"out": torch.cat(parts)}


# ------------------------------------------------------------------------------------------------ the package's calls

def _own(st):
    import chunked_prefill_mixed_decode_gb300 as ms
    if st["op"] == "tables":
        ms.build_batch_metadata_device(st["cached"], st["new"], st["tables"], st["pages"], st["cu"], st["start"], st["ctx"],
                                       st["positions"], st["slots"], block_tables=st["bt"], bt_offsets=st["bt_offsets"],
                                       bt_pages=st["bt_pages"], free_pages=st["free"], free_count=st["free_count"],
                                       free_state=st["free_state"], info=st["info"])
        out = {"cu": st["cu"], "start": st["start"], "ctx": st["ctx"], "positions": st["positions"], "slots": st["slots"],
               "tables": st["tables"], "free_count": st["free_state"][:1], "info": st["info"]}
        return out | ({"bt_offsets": st["bt_offsets"], "bt_pages": st["bt_pages"]} if st["ragged"] else {"bt": st["bt"]})
    if st["op"] == "append":
        ms.kv_append_rope_q4(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["cos"], st["sin"], st["pool"],
                             q_rot=st["q_rot"])
        ms.kv_read_q4(st["pool"], st["slots"], st["k_out"], st["v_out"])
        return {"q_rot": st["q_rot"], "k": st["k_out"], "v": st["v_out"]}
    if st["op"] == "read":
        ms.kv_read_q4(st["pool"], st["slots"], st["k_out"], st["v_out"])
        return {"k": st["k_out"], "v": st["v_out"]}
    if "workspace" not in st:  # kept by the caller for all its steps
        n = ms.attention_workspace_size(st["ctx"].numel(), st["q_rot"].shape[0], st["context_total"], st["H_q"], st["H_kv"], st["D"])
        st["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    ms.mixed_step_attention_q4(st["q_rot"], st["pool"], st["cu"], st["start"], st["ctx"],
                               st["bt_pages"] if st["ragged"] else st["bt"], st["context_total"], st["out"], st["workspace"],
                               bt_offsets=st["bt_offsets"] if st["ragged"] else None)
    return {"out": st["out"]}


def run(state):
    if own:
        return _own(state)
    return {"tables": _plain_tables, "append": _plain_append, "read": _plain_read, "attend": _plain_attend}[state["op"]](state)


# ------------------------------------------------------------------------------------------------ in 64 bits

def _where(D):
    """Byte and shift of element d of row r in a block, for K and for V, as index arrays [16, D]."""
    r, d = torch.arange(PAGE)[:, None], torch.arange(D)[None]
    g, e = d // GROUP, d % GROUP
    lane, i, odd = e // 8, (e % 8) // 2, e % 2
    NG = D // GROUP
    k = r * D + (lane * NG + g) * 8 + odd * 4 + i          # in nibbles
    v = PAGE * D + r * D + ((lane * 2 + odd) * NG + g) * 4 + i
    return [(x // 2, (x % 2) * 4) for x in (k, v)]


def _values64(pool, pages, D, which):
    """K (which 0) or V (1) rows [len(pages), H, 16, D] in 64 bits."""
    byte, shift = (x.to(pool.device) for x in _where(D)[which])
    b = pool[pages]
    NG = D // GROUP
    code = ((b[..., byte.reshape(-1)] >> shift.reshape(-1).to(torch.uint8)) & 15).double() - 8.0
    lo = 16 * D + which * PAGE * NG * 2
    bits = b[..., lo: lo + PAGE * NG * 2].to(torch.int32)
    s = ((bits[..., 0::2] << 16) | (bits[..., 1::2] << 24)).contiguous().view(torch.float32).double()
    code = code.view(*b.shape[:2], PAGE, D)
    return code * s.view(*b.shape[:2], PAGE, NG).repeat_interleave(GROUP, dim=-1)


def _held64(x):
    """The values that a row stands for once it is held in 4 bits."""
    g = x.view(*x.shape[:-1], -1, GROUP)
    m, e = torch.frexp(g.abs().max(dim=-1, keepdim=True).values / 7.0)
    s = torch.ldexp(torch.round(m * 32.0) / 32.0, e)
    return (s * torch.round(g / s)).view(x.shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "tables":
        return None  # whole numbers
    D = st["D"]
    if case["op"] == "read":
        slot = st["slots"].long()
        every = [_values64(st["pool"], slice(None), D, w) for w in (0, 1)]
        return {"k": every[0][slot // PAGE, :, slot % PAGE], "v": every[1][slot // PAGE, :, slot % PAGE]}
    if case["op"] == "append":
        cos, sin = (st[n].double()[st["positions"].long()].unsqueeze(1) for n in ("cos", "sin"))

        def turn(x):
            y = x.double()
            h = D // 2
            return torch.cat([y[..., :h] * cos - y[..., h:] * sin, y[..., h:] * cos + y[..., :h] * sin], dim=-1)

        return {"q_rot": turn(st["q"]), "k": _held64(turn(st["k"]).to(torch.bfloat16).double()), "v": _held64(st["v"].double())}
    H_q, H_kv = st["H_q"], st["H_kv"]
    G = H_q // H_kv
    out = torch.empty((st["q_rot"].shape[0], H_q, D), dtype=torch.float64, device="cuda")
    cu, start, offs = st["cu"].tolist(), st["start"].tolist(), st["bt_offsets"].tolist()
    for r in range(len(start)):
        pages = st["bt_pages"][offs[r]: offs[r + 1]].long()
        d = cu[r + 1] - cu[r]
        n = start[r] + d
        K, V = (_values64(st["pool"], pages, D, w).transpose(0, 1).reshape(H_kv, -1, D)[:, :n] for w in (0, 1))
        seen = torch.arange(n, device="cuda")[None] <= start[r] + torch.arange(d, device="cuda")[:, None]
        for h in range(H_kv if d > 1 else 1):
            if d > 1:  # one KV head at a time
                q = st["q_rot"][cu[r]: cu[r + 1], h * G: (h + 1) * G].double().permute(1, 0, 2)
                p = torch.softmax(torch.where(seen, q @ K[h].T / math.sqrt(D), -math.inf), dim=-1)
                out[cu[r]: cu[r + 1], h * G: (h + 1) * G] = (p @ V[h]).permute(1, 0, 2)
            else:
                q = st["q_rot"][cu[r]].double().view(H_kv, G, D)
                p = torch.softmax(q @ K.transpose(1, 2) / math.sqrt(D), dim=-1)
                out[cu[r]] = (p @ V).reshape(H_q, D)
    return {"out": out}
