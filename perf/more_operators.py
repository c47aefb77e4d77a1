"""Attention steps of models with other rotations and other views of the cache: plain forms, and the package's calls.

Four operators make such a step:

* table  -- the rotary table of a run of positions, with the frequencies scaled for long contexts, on the GPU;
* append -- the rotary embedding over part of the head, in pairs (i, i + R/2) or (2i, 2i + 1), and the paged append of
  K and V, from rows of a fused projection; without rotation and without q for an encoder's states;
* window -- causal attention of every packed row over the last W keys of its pages, with an optional sink: one more
  logit per head in the softmax's sum, without a value;
* cross  -- attention of every packed row to all of an encoder's states in its pages, of another length.

Pages hold 16 tokens: [pages, H_kv, 16, D], bf16.
"""
import math
import random

import torch

own = False

PAGE = 16


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the table of a 16K context, frequencies as they are
        {"name": "table_plain_16k", "op": "table", "rows": 16384, "first": 0, "R": 128, "base": 10000.0, "kind": "plain",
         "factor": 1.0, "original": 16384},
        # the table of a 128K context from frequencies that were trained to 32K, scaled by a ramp over the dimensions
        {"name": "table_ramp_128k", "op": "table", "rows": 131072, "first": 0, "R": 128, "base": 10000.0, "kind": "ramp",
         "factor": 4.0, "original": 32768},
        # a decode-only step of 64 requests, 32 KV heads: half of each head turned in neighbouring pairs
        {"name": "append_decode_64", "op": "append", "tokens": 64, "H_q": 32, "H_kv": 32, "D": 128, "R": 64,
         "interleaved": True, "ctx_hi": 4096, "fused": True},
        # a full mixed step with grouped heads, rows of a fused projection, part of the head turned in halves
        {"name": "append_mixed_8192", "op": "append", "tokens": 8192, "H_q": 32, "H_kv": 8, "D": 128, "R": 64,
         "interleaved": False, "ctx_hi": 16384, "fused": True},
        # an encoder's states of 6000 positions put into pages: no query, no rotation
        {"name": "append_states_6000", "op": "append", "tokens": 6000, "H_q": 0, "H_kv": 8, "D": 128, "R": 0,
         "interleaved": False, "ctx_hi": 16384, "fused": False},
        # the smallest step: three short decodes and a 5-token chunk, where the latency of a call counts
        {"name": "window_small_8", "op": "window", "H_q": 4, "H_kv": 2, "D": 64, "decodes": 3, "ctx_lo": 37, "ctx_hi": 100,
         "chunks": 1, "chunk_tokens": 5, "chunk_start": 0, "chunk_step": 0, "ragged": False, "window": 32, "sinks": True,
         "released": False},
        # decodes of a grouped-query layer that sees 1024 keys: 256 requests of 700 to 16K tokens, older pages given back
        {"name": "window_decode_gqa_256", "op": "window", "H_q": 32, "H_kv": 8, "D": 128, "decodes": 256, "ctx_lo": 700,
         "ctx_hi": 16384, "chunks": 0, "chunk_tokens": 0, "chunk_start": 0, "chunk_step": 0, "ragged": True,
         "window": 1024, "sinks": False, "released": True},
        # prompt chunks alone, at the start and far into a prompt, 1024 keys each
        {"name": "window_chunk_gqa_2", "op": "window", "H_q": 32, "H_kv": 8, "D": 128, "decodes": 0, "ctx_lo": 1,
         "ctx_hi": 1, "chunks": 2, "chunk_tokens": 3968, "chunk_start": 0, "chunk_step": 6000, "ragged": False,
         "window": 1024, "sinks": False, "released": False},
        # odd sizes, eight query heads to a KV head, half the head dim, a short window with sinks
        {"name": "window_odd_d64", "op": "window", "H_q": 16, "H_kv": 2, "D": 64, "decodes": 61, "ctx_lo": 1,
         "ctx_hi": 5003, "chunks": 3, "chunk_tokens": 777, "chunk_start": 11, "chunk_step": 1501, "ragged": True,
         "window": 128, "sinks": True, "released": True},
        # the largest: long decodes next to the last chunk of a 32K prompt, 4096 keys each
        {"name": "window_mixed_long", "op": "window", "H_q": 32, "H_kv": 8, "D": 128, "decodes": 16, "ctx_lo": 65536,
         "ctx_hi": 131072, "chunks": 1, "chunk_tokens": 4096, "chunk_start": 28672, "chunk_step": 0, "ragged": True,
         "window": 4096, "sinks": False, "released": True},
        # one new token each of 64 requests over their encoder states of 300 to 1500 positions, three without any
        {"name": "cross_decode_64", "op": "cross", "H_q": 32, "H_kv": 32, "D": 128, "decodes": 64, "ctx_lo": 300,
         "ctx_hi": 1500, "empty": 3, "chunks": 0, "chunk_tokens": 0, "chunk_keys": 0, "chunk_step": 0, "ragged": False},
        # two prompts of 512 tokens over 6000 and 5000 states, grouped heads
        {"name": "cross_chunk_gqa_2", "op": "cross", "H_q": 32, "H_kv": 8, "D": 128, "decodes": 0, "ctx_lo": 1,
         "ctx_hi": 1, "empty": 0, "chunks": 2, "chunk_tokens": 512, "chunk_keys": 6000, "chunk_step": -1000,
         "ragged": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "append", "append", "window", "window", "window", "cross", "cross"])
    if op == "table":
        rows = _log(rng, 1, 131072)
        return {"op": op, "rows": rows, "first": rng.choice([0, _log(rng, 1, 1000000)]), "R": rng.choice([16, 32, 48, 64, 96, 128]),
                "base": rng.choice([10000.0, 500000.0, 1000000.0]), "kind": rng.choice(["plain", "linear", "base", "bands", "ramp"]),
                "factor": rng.choice([1.5, 2.0, 4.0, 8.0, 32.0]), "original": rng.choice([2048, 4096, 8192, 32768])}
    G = rng.choice([1, 2, 4, 8])
    H_kv = rng.choice([1, 2, 4, 8, 10] if G > 2 else [2, 8, 16, 32, 40])
    H_q, D = G * H_kv, rng.choice([64, 128])
    if op == "append":
        R = 16 * rng.randint(0, D // 16)
        return {"op": op, "tokens": _log(rng, 1, 8192), "H_q": H_q if rng.random() < 0.8 else 0, "H_kv": H_kv, "D": D, "R": R,
                "interleaved": rng.random() < 0.5, "ctx_hi": _log(rng, 64, 16384), "fused": rng.random() < 0.5}
    rows = _log(rng, 1, 256)
    chunks = rng.choice([0, 1, 1, 2, 3])
    d = _log(rng, 2, 4096 // max(1, chunks)) if chunks else 0
    c = {"op": op, "H_q": H_q, "H_kv": H_kv, "D": D, "decodes": rows, "chunks": chunks, "ragged": rng.random() < 0.5}
    if op == "cross":
        hi = _log(rng, 1, min(6000, max(16, 2_000_000 // rows // H_kv)))
        keys = _log(rng, 1, 6000) if chunks else 0
        d = max(2, min(d, 4096 * 4096 * 32 // max(1, chunks * keys * H_q))) if chunks else 0
        return {**c, "ctx_lo": rng.randint(1, hi), "ctx_hi": hi, "empty": rng.choice([0, 0, 1, rows]) if rows > 1 else 0,
                "chunk_tokens": d, "chunk_keys": keys, "chunk_step": -rng.randint(0, keys // 2) if chunks else 0}
    window = _log(rng, 1, min(8192, max(16, 2_000_000 // rows // H_kv)))
    hi = _log(rng, 16, 131072)
    released = rng.random() < 0.6
    if not released:
        hi = min(hi, max(16, 4_000_000 // rows // H_kv))
    start = rng.choice([0, _log(rng, 1, 28672)]) if chunks else 0
    d = max(2, min(d, 4096 * 4096 * 32 // max(1, chunks * window * H_q))) if chunks else 0
    return {**c, "ctx_lo": rng.randint(1, hi), "ctx_hi": hi, "chunk_tokens": d, "chunk_start": start,
            "chunk_step": rng.randint(0, 2000) if chunks else 0, "window": window, "sinks": rng.random() < 0.5, "released": released}


def _rows(case):
    """(c, d) of every row of a window case: the decodes' lengths spaced evenly over their logarithm, then the chunks."""
    n, lo, hi = case["decodes"], case["ctx_lo"], case["ctx_hi"]
    dec = [(int(round(lo * (hi / lo) ** (i / max(1, n - 1)))), 1) for i in range(n)]
    return dec + [(case["chunk_start"] + i * case["chunk_step"], case["chunk_tokens"]) for i in range(case["chunks"])]


def _cross_rows(case):
    """(keys, d) of every row of a cross case; `empty` of the decodes have no keys."""
    n, lo, hi = case["decodes"], case["ctx_lo"], case["ctx_hi"]
    dec = [(0 if i < case["empty"] else int(round(lo * (hi / lo) ** (i / max(1, n - 1)))), 1) for i in range(n)]
    return dec + [(case["chunk_keys"] + i * case["chunk_step"], case["chunk_tokens"]) for i in range(case["chunks"])]


def _pages(n):
    return (n + PAGE - 1) // PAGE


def _first(c, window):
    """The first key that a row of c cached tokens sees."""
    return max(0, c + 1 - window)


def work(case):
    if case["op"] == "table":
        pairs = case["rows"] * case["R"] // 2
        return {"bytes": 8 * pairs, "flops": 8 * pairs}  # cos and sin, fp32
    H_q, H_kv, D = case["H_q"], case["H_kv"], case["D"]
    if case["op"] == "append":
        T, R = case["tokens"], case["R"]
        return {"bytes": T * (4 * H_q * D + 8 * H_kv * D + 4 * R + 8), "flops": 3 * T * (H_q + H_kv) * R}
    if case["op"] == "cross":
        rows = _cross_rows(case)
        kv = sum(n for n, _ in rows)
        pairs = sum(n * d for n, d in rows)
        pages = sum(_pages(n) for n, _ in rows)
    else:
        rows, W = _rows(case), case["window"]
        kv = sum(c + d - _first(c, W) for c, d in rows)
        pages = sum(_pages(c + d) - _first(c, W) // PAGE for c, d in rows)
        pairs = 0
        for c, d in rows:
            low = max(0, min(d, W - c))  # tokens that see everything before them
            pairs += low * c + low * (low + 1) // 2 + (d - low) * W
    T = sum(d for _, d in rows)
    return {"bytes": kv * H_kv * D * 4 + 4 * T * H_q * D + 4 * (pages + 4 * len(rows)), "flops": 4 * D * H_q * pairs}


# ------------------------------------------------------------------------------------------------ inputs

def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _frequencies(case):
    """The angle per position of every pair, and what cosine and sine are multiplied by."""
    R, base, kind, s, n = case["R"], case["base"], case["kind"], case["factor"], case["original"]
    if kind == "base":
        base = base * s ** (R / (R - 2))
    f = [base ** (-2.0 * i / R) for i in range(R // 2)]
    if kind == "linear":
        return [x / s for x in f], 1.0
    if kind == "bands":  # wavelengths longer than n are stretched, those shorter than n / 4 are not
        g = []
        for x in f:
            t = min(1.0, max(0.0, (n * x / (2 * math.pi) - 1.0) / (4.0 - 1.0)))
            g.append((1.0 - t) * x / s + t * x)
        return g, 1.0
    if kind == "ramp":  # pairs that turn 32 times over n are not stretched, those that turn less than once are
        at = lambda turns: R * math.log(n / (turns * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), R - 1)
        hi = hi + 0.001 if hi == lo else hi
        t = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(R // 2)]
        return [x / s * a + x * (1.0 - a) for x, a in zip(f, t)], 0.1 * math.log(s) + 1.0
    return f, 1.0


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    randn = lambda *shape: torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    if case["op"] == "table":
        first = case["first"] + seed % 977  # where the run starts moves with the seed
        return {**case, "first": first, "cos": torch.empty((case["rows"], case["R"] // 2), device="cuda"),
                "sin": torch.empty((case["rows"], case["R"] // 2), device="cuda")}
    H_q, H_kv, D = case["H_q"], case["H_kv"], case["D"]
    if case["op"] == "append":
        T, R = case["tokens"], case["R"]
        pages = _pages(2 * T)
        slots = torch.randperm(PAGE * pages, generator=gen, device="cuda")[:T].to(torch.int32)
        pos = torch.randint(0, case["ctx_hi"], (T,), generator=gen, device="cuda", dtype=torch.int32)
        if case["fused"]:  # q, k and v of a token side by side, as one projection leaves them
            q, k, v = randn(T, H_q + 2 * H_kv, D).split([H_q, H_kv, H_kv], dim=1)
        else:
            q, k, v = (randn(T, n, D) for n in (H_q, H_kv, H_kv))
        st = {**case, "q": q if H_q else None, "k": k, "v": v, "positions": pos, "slots": slots, "cos": None, "sin": None,
              "k_cache": torch.zeros((pages, H_kv, PAGE, D), dtype=torch.bfloat16, device="cuda"),
              "v_cache": torch.zeros((pages, H_kv, PAGE, D), dtype=torch.bfloat16, device="cuda"),
              "q_rot": torch.empty((T, H_q, D), dtype=torch.bfloat16, device="cuda") if H_q else None}
        if R:
            freq = 10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
            ang = torch.arange(case["ctx_hi"], device="cuda", dtype=torch.float64)[:, None] * freq
            st.update(cos=ang.cos().float(), sin=ang.sin().float())
        return st
    cross = case["op"] == "cross"
    rows = _cross_rows(case) if cross else _rows(case)
    dec = rows[: case["decodes"]]
    r.shuffle(dec)
    rows = dec + rows[case["decodes"]:]
    ends = [n if cross else n + d for n, d in rows]
    need = [_pages(n) for n in ends]
    gone = [0 if cross or not case["released"] else _first(c, case["window"]) // PAGE for c, _ in rows]
    held = sum(n - g for n, g in zip(need, gone))
    T, R, stride, total = sum(d for _, d in rows), len(rows), max(1, max(need)), sum(need)
    # a row's pages in order; those in front of its window have been given back and their entries say nothing
    ids = torch.randperm(max(1, held), generator=gen, device="cuda").to(torch.int32)
    off = [0]
    for n in need:
        off.append(off[-1] + n)
    offs, goneT = _ints(off), _ints(gone)
    row = torch.repeat_interleave(torch.arange(R, device="cuda"), _ints(need).long(), output_size=total)
    j = torch.arange(total, device="cuda") - offs[row].long()
    kept = j >= goneT[row]
    flat = torch.full((max(1, total),), -1, dtype=torch.int32, device="cuda")
    if held:
        flat[:total][kept] = ids[: held]
    bt = torch.full((R, stride), -1, dtype=torch.int32, device="cuda")
    if total:
        bt[row, j] = flat[:total]
    cu = [0]
    for _, d in rows:
        cu.append(cu[-1] + d)
    st = {**case, "q": randn(T, H_q, D), "k_cache": randn(max(1, held), H_kv, PAGE, D), "v_cache": randn(max(1, held), H_kv, PAGE, D),
          "cu": _ints(cu), "ends": _ints(ends), "bt": bt, "bt_offsets": offs, "bt_pages": flat, "total": sum(ends), "rows": rows,
          "out": torch.empty((T, H_q, D), dtype=torch.bfloat16, device="cuda"), "sink": None}
    if not cross:
        st["start"] = _ints([c for c, _ in rows])
        if case["sinks"]:
            st["sink"] = 2.0 * torch.randn(H_q, generator=gen, device="cuda")
    return st


# ------------------------------------------------------------------------------------------------ plain forms

def _plain_table(st):
    f, amp = _frequencies(st)
    pos = torch.arange(st["first"], st["first"] + st["rows"], device="cuda", dtype=torch.float64)
    ang = pos[:, None] * torch.tensor(f, device="cuda", dtype=torch.float64)
    return {"cos": (ang.cos() * amp).float(), "sin": (ang.sin() * amp).float()}


def _plain_turn(x, st):
    R = st["R"]
    if R == 0:
        return x
    cos, sin = (st[n][st["positions"].long()][:, None] for n in ("cos", "sin"))
    y = x[..., :R].float()
    if st["interleaved"]:
        a, b = y[..., 0::2], y[..., 1::2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y.chunk(2, dim=-1)
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y.to(torch.bfloat16), x[..., R:]], -1)


def _plain_append(st):
    page, at = st["slots"].long() // PAGE, st["slots"].long() % PAGE
    st["k_cache"][page, :, at] = _plain_turn(st["k"], st)
    st["v_cache"][page, :, at] = st["v"]
    out = {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    return out if st["q"] is None else {**out, "q_rot": _plain_turn(st["q"], st)}


def _plain_rows(st, r0, r1, t0, d, first, keys, low, high):
    """Rows r0..r1-1, d tokens each from token t0 on, over `keys` keys of their pages from key first[row] (a multiple of
    16) on; token i of a row sees keys low[row, i] to high[row, i] - 1."""
    H_q, H_kv, D, R, P = st["H_q"], st["H_kv"], st["D"], r1 - r0, max(1, _pages(keys))
    G, dev = H_q // H_kv, st["q"].device
    page = (first[:, None] // PAGE + torch.arange(P, device=dev)).clamp(max=st["bt"].shape[1] - 1)
    ids = st["bt"][r0:r1].long().gather(1, page).clamp(min=0)
    key = first[:, None] + torch.arange(P * PAGE, device=dev)
    hidden = (key[:, None] < low[..., None]) | (key[:, None] >= high[..., None])  # [R, d, keys]
    out = torch.empty((R * d, H_q, D), dtype=torch.bfloat16, device=dev)
    q = st["q"][t0: t0 + R * d].view(R, d, H_kv, G, D).permute(0, 2, 3, 1, 4)
    step = 1 if R * d * G * P * PAGE > 1 << 26 else H_kv  # KV heads at a time
    for h in range(0, H_kv, step):
        k, v = (st[n][ids, h: h + step].transpose(1, 2).reshape(R, step, P * PAGE, D).float() for n in ("k_cache", "v_cache"))
        s = torch.matmul(q[:, h: h + step].float().reshape(R, step, G * d, D), k.transpose(-1, -2))
        s = (s * D ** -0.5).view(R, step, G, d, P * PAGE).masked_fill_(hidden[:, None, None], -math.inf)
        m = s.amax(-1, keepdim=True)
        if st["sink"] is not None:
            sink = st["sink"][h * G: (h + step) * G].view(1, step, G, 1, 1)
            m = torch.maximum(m, sink)
        m = torch.where(m == -math.inf, 0.0, m)  # a row that sees no key
        p = torch.exp(s - m)
        total = p.sum(-1, keepdim=True)
        if st["sink"] is not None:
            total = total + torch.exp(sink - m)
        o = torch.matmul(p.view(R, step, G * d, P * PAGE), v).view(R, step, G, d, D)
        o = torch.where(total > 0, o / total, 0.0)
        out.view(R, d, H_q, D)[:, :, h * G: (h + step) * G] = o.permute(0, 3, 1, 2, 4).reshape(R, d, step * G, D).to(torch.bfloat16)
    return out


def _plain_attend(st):
    n, m, cross = st["decodes"], st["chunks"], st["op"] == "cross"
    parts = []
    for r0, r1, t0, d in [(0, n, 0, 1)] * (n > 0) + [(n + i, n + i + 1, n + i * st["chunk_tokens"], st["chunk_tokens"]) for i in range(m)]:
        high = st["ends"][r0:r1].long()[:, None].expand(-1, d)
        if cross:
            low = first = torch.zeros_like(high)
            keys = max(k for k, _ in st["rows"][r0:r1])
        else:
            high = st["start"][r0:r1].long()[:, None] + 1 + torch.arange(d, device="cuda")
            low = (high - st["window"]).clamp(min=0)
            first = low // PAGE * PAGE
            keys = max(c + k - _first(c, st["window"]) // PAGE * PAGE for c, k in st["rows"][r0:r1])
        parts.append(_plain_rows(st, r0, r1, t0, d, first[:, 0], keys, low, high))
    return {"out": torch.cat(parts)}


# ------------------------------------------------------------------------------------------------ the package's calls

def _scaling(st):
    kind = st["kind"]
    if kind == "plain":
        return None
    s = {"kind": kind, "factor": st["factor"]}
    if kind == "bands":
        s.update(original_len=st["original"], low=1.0, high=4.0)
    if kind == "ramp":
        s.update(original_len=st["original"], low=1.0, high=32.0)
    return s


def _own(st):
    import chunked_prefill_mixed_decode_gb300 as ms
    if st["op"] == "table":
        freq, amplitude = ms.rotary_frequencies(st["R"], st["base"], _scaling(st))
        ms.rotary_table_device(freq, st["cos"], st["sin"], amplitude=amplitude, first_pos=st["first"])
        return {"cos": st["cos"], "sin": st["sin"]}
    if st["op"] == "append":
        ms.kv_append_rotary(st["q"], st["k"], st["v"], st["positions"], st["slots"], st["cos"], st["sin"], st["k_cache"],
                            st["v_cache"], q_rot=st["q_rot"], interleaved=st["interleaved"])
        out = {"k_cache": st["k_cache"], "v_cache": st["v_cache"]}
        return out if st["q"] is None else {**out, "q_rot": st["q_rot"]}
    if "workspace" not in st:  # kept by the caller for all its steps
        n = ms.attention_workspace_size(len(st["rows"]), st["q"].shape[0], st["total"], st["H_q"], st["H_kv"], st["D"])
        st["workspace"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    table, offsets = (st["bt_pages"], st["bt_offsets"]) if st["ragged"] else (st["bt"], None)
    if st["op"] == "cross":
        ms.mixed_step_cross_attention(st["q"], st["k_cache"], st["v_cache"], st["cu"], st["ends"], table, st["total"], st["out"],
                                      st["workspace"], bt_offsets=offsets)
    else:
        ms.mixed_step_attention_window(st["q"], st["k_cache"], st["v_cache"], st["cu"], st["start"], st["ends"], table,
                                       st["total"], st["out"], st["workspace"], st["window"], sinks=st["sink"],
                                       bt_offsets=offsets)
    return {"out": st["out"]}


def run(state):
    if own:
        return _own(state)
    return {"table": _plain_table, "append": _plain_append, "window": _plain_attend, "cross": _plain_attend}[state["op"]](state)


# ------------------------------------------------------------------------------------------------ in 64 bits

def _exact_table(st):
    R, n = st["R"], st["original"]
    base = st["base"] * st["factor"] ** (R / (R - 2.0)) if st["kind"] == "base" else st["base"]
    i = torch.arange(R // 2, dtype=torch.float64)
    f = torch.exp(-(2.0 * i / R) * math.log(base))
    amp = 1.0
    if st["kind"] == "linear":
        f = f / st["factor"]
    elif st["kind"] == "bands":
        wave = 2.0 * math.pi / f
        keep = ((n / wave - 1.0) / 3.0).clamp(0.0, 1.0)
        f = torch.lerp(f / st["factor"], f, keep)
    elif st["kind"] == "ramp":
        def dim(turns):  # the pair that turns so often over n positions
            return 0.5 * R * (math.log(n) - math.log(2.0 * math.pi * turns)) / math.log(base)

        lo, hi = float(max(0, math.floor(dim(32.0)))), float(min(R - 1, math.ceil(dim(1.0))))
        hi += 0.001 * (hi == lo)
        f = torch.lerp(f, f / st["factor"], ((i - lo) / (hi - lo)).clamp(0.0, 1.0))
        amp += 0.1 * math.log(st["factor"])
    ang = torch.outer(torch.arange(st["rows"], dtype=torch.float64, device="cuda") + float(st["first"]), f.cuda())
    return {"cos": amp * torch.cos(ang), "sin": amp * torch.sin(ang)}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "table":
        return _exact_table(st)
    if case["op"] == "append":
        R, slot = st["R"], st["slots"].long()

        def turn(x):
            y = x.double().clone()
            if R:
                i = torch.arange(R // 2, device="cuda")
                a, b = (2 * i, 2 * i + 1) if st["interleaved"] else (i, i + R // 2)
                z = torch.complex(y[..., a], y[..., b])
                w = torch.complex(st["cos"].double(), st["sin"].double()).index_select(0, st["positions"].long()).unsqueeze(1)
                z = z * w
                y[..., a], y[..., b] = z.real, z.imag
            return y

        out = {}
        for name, x in (("k_cache", turn(st["k"])), ("v_cache", st["v"].double())):
            pool = st[name].double().permute(0, 2, 1, 3).reshape(-1, st["H_kv"], st["D"])
            pool[slot] = x
            out[name] = pool.view(-1, PAGE, st["H_kv"], st["D"]).permute(0, 2, 1, 3).contiguous()
        if st["q"] is not None:
            out["q_rot"] = turn(st["q"])
        return out
    H_q, H_kv, D = st["H_q"], st["H_kv"], st["D"]
    G, cross = H_q // H_kv, case["op"] == "cross"
    out = torch.zeros((st["q"].shape[0], H_q, D), dtype=torch.float64, device="cuda")
    offs, t0 = st["bt_offsets"].tolist(), 0
    for r, (c, d) in enumerate(st["rows"]):
        n = c if cross else c + d
        lo = 0 if cross else _first(c, st["window"]) // PAGE
        pages = st["bt_pages"][offs[r] + lo: offs[r + 1]].long()
        t1 = t0 + d
        if n > 0:
            K, V = (st[name][pages].double().transpose(0, 1).reshape(H_kv, -1, D)[:, : n - lo * PAGE] for name in ("k_cache", "v_cache"))
            j = torch.arange(lo * PAGE, n, device="cuda")
            p = torch.arange(c, c + d, device="cuda")[:, None]
            seen = torch.ones((d, j.numel()), dtype=torch.bool, device="cuda") if cross else (j <= p) & (j > p - st["window"])
            step = 1 if d > 1 else H_kv  # KV heads at a time
            for h in range(0, H_kv, step):
                q = st["q"][t0:t1, h * G: (h + step) * G].double().view(d, step, G, D).permute(1, 2, 0, 3)
                s = torch.where(seen, q @ K[h: h + step, None].transpose(2, 3) / math.sqrt(D), -math.inf)
                if st["sink"] is not None:  # a last key with the sink's score and a value of zero
                    s = torch.cat([s, st["sink"][h * G: (h + step) * G].double().view(step, G, 1, 1).expand(-1, -1, d, 1)], -1)
                w = torch.softmax(s, -1)[..., : j.numel()]
                out[t0:t1, h * G: (h + step) * G] = (w @ V[h: h + step, None]).permute(2, 0, 1, 3).reshape(d, step * G, D)
        t0 = t1
    return {"out": out}
