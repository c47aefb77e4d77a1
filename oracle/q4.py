"""Oracle: the 4-bit K/V cache -- its rounding, its bytes, and the metadata of a step built from lengths.

The rounding, per group of 32 consecutive elements of a row, with a = max |x|:

    s = r5(a / 7),  code = rint(x / s),  value = s * code

r5 keeps five significant bits (nearest, ties to even).  A group whose a / 7 is
below 2**-126 is stored as zeros, s is at most 1.125 * 2**125, and a group with
an infinity or a NaN is stored as zeros.

The bytes of one page of one KV head, 18 D of them: 16 K rows and 16 V rows of
D / 2 bytes of nibbles (code + 8), then the K scales and the V scales as bf16
[16][D / 32].  The pages on chunked prefill have no counterpart; attention over
such a cache is attention over the values that it holds.
"""
from __future__ import annotations

import numpy as np

GROUP = 32
PAGE = 16


def q4_round(x):
    """Rows x [..., D] (fp64) -> codes [..., D] (int64) and scales [..., D/32] (fp64)."""
    x = np.asarray(x, dtype=np.float64)
    g = x.reshape(x.shape[:-1] + (-1, GROUP))
    ok = np.isfinite(g).all(axis=-1)
    g = np.where(ok[..., None], g, 0.0)
    r = np.abs(g).max(axis=-1) / 7.0
    m, e = np.frexp(r)  # r = m 2^e, m in [1/2, 1): 32 m has five bits before the point
    s = np.ldexp(np.round(m * 32.0), e - 5)
    s = np.where(r < 2.0 ** -126, 0.0, np.minimum(s, 1.125 * 2.0 ** 125))
    codes = np.round(np.divide(g, s[..., None], out=np.zeros_like(g), where=s[..., None] > 0))
    return codes.astype(np.int64).reshape(x.shape), s


def q4_values(x):
    """The values that rows x stand for once they are held in 4 bits."""
    codes, s = q4_round(x)
    return codes * np.repeat(s, GROUP, axis=-1)


def nibble_index(D, d, is_v):
    """Place of element d of a row, in nibbles from the row's start."""
    NG = D // GROUP
    g, t, e = d // GROUP, (d % GROUP) // 8, d % 8
    if is_v:
        return ((2 * t + e % 2) * NG + g) * 4 + e // 2
    return (t * NG + g) * 8 + (e % 2) * 4 + e // 2


def q4_write(pool, slot, head, x, is_v):
    """Store one row x [D] (fp64) at a slot of a pool [pages, H, 18 D] of uint8 (in place)."""
    D = x.shape[-1]
    NG = D // GROUP
    codes, s = q4_round(x)
    blk = pool[slot // PAGE, head]
    row = slot % PAGE
    base = (PAGE * D // 2 if is_v else 0) + row * D // 2
    out = np.zeros(D // 2, dtype=np.uint8)
    for d in range(D):
        n = nibble_index(D, d, is_v)
        out[n // 2] |= np.uint8((int(codes[d]) + 8) << (4 * (n % 2)))
    blk[base:base + D // 2] = out
    sb = (np.asarray(s, dtype=np.float32).view(np.uint32) >> 16).astype(np.uint16)  # exact: five bits
    at = PAGE * D + (PAGE * NG * 2 if is_v else 0) + row * NG * 2
    blk[at:at + NG * 2] = sb.view(np.uint8)


def q4_read(pool, D):
    """The K and V values of a pool [..., 18 D]: two arrays [..., 16, D] (fp64)."""
    NG = D // GROUP
    lead = pool.shape[:-1]
    out = []
    for w in (0, 1):
        b = pool[..., w * PAGE * D // 2:(w + 1) * PAGE * D // 2].reshape(lead + (PAGE, D // 2))
        n = np.array([nibble_index(D, d, w == 1) for d in range(D)])
        codes = ((b[..., n // 2] >> (4 * (n % 2)).astype(np.uint8)) & 15).astype(np.float64) - 8.0
        at = PAGE * D + w * PAGE * NG * 2
        sb = np.ascontiguousarray(pool[..., at:at + PAGE * NG * 2]).view(np.uint16).astype(np.uint32) << 16
        s = sb.view(np.float32).astype(np.float64).reshape(lead + (PAGE, NG))
        out.append(codes * np.repeat(s, GROUP, axis=-1))
    return out


def metadata_from_lengths(cached, new, tables, cap_tokens, free=None, count=0):
    """The step's metadata from the requests' lengths: row s is request s with cached[s] tokens and new[s] new ones.

    Returns a dict; ``tables`` [rows, stride] is copied and the pages taken from the end of ``free`` entered.
    """
    tables = np.array(tables, dtype=np.int64)
    cu, start, ctx, positions, slots, pages, offs = [0], [], [], [], [], [], [0]
    taken = 0
    for s, (c, d) in enumerate(zip(cached, new)):
        c, d = int(c), int(d)
        n = -(-(c + d) // PAGE) if d else 0
        if free is not None:
            for j in range(-(-c // PAGE), n):
                tables[s, j] = free[count - 1 - taken]
                taken += 1
        cu.append(cu[-1] + d)
        start.append(c if d else 0)
        ctx.append(c + d if d else 0)
        for p in range(c, c + d):
            positions.append(p)
            slots.append(int(tables[s, p // PAGE]) * PAGE + p % PAGE)
        pages += [int(x) for x in tables[s, :n]]
        offs.append(len(pages))
    pad = cap_tokens - len(positions)
    return {"cu_seqlens_q": cu, "q_start_pos": start, "context_lens": ctx, "positions": positions + [0] * pad,
            "slot_mapping": slots + [-1] * pad, "bt_offsets": offs, "bt_pages": pages, "tables": tables,
            "free_count": count - taken,
            "info": [cu[-1], len(pages), sum(1 for d in new if d == 1), taken]}
