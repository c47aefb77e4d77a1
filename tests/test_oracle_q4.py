"""The 4-bit cache on the CPU: pins of the oracle's rounding, bytes and metadata, and the
argument checks of the calls."""
import numpy as np
import pytest

import oracle


def _bf16(rng, shape, sigma=1.0):
    x = (rng.standard_normal(shape) * sigma).astype(np.float32)
    return oracle.bf16_to_f64(oracle.f32_to_bf16_bits(x))


def test_values_are_bf16_and_within_half_a_step():
    """Every value is exactly a bf16 (a scale of 5 bits times a code of 3), and no element is further than
    half a step from its own: |x| <= 7 s (1 + 2^-5), so nothing is clipped."""
    rng = np.random.default_rng(1)
    for sigma in (1e-30, 1e-3, 1.0, 7.0, 1e30):
        x = _bf16(rng, (200, 128), sigma)
        codes, s = oracle.q4_round(x)
        v = oracle.q4_values(x)
        assert codes.min() >= -7 and codes.max() <= 7
        assert np.array_equal(oracle.bf16_to_f64(oracle.f32_to_bf16_bits(v.astype(np.float32))), v)
        assert (np.abs(v - x) <= np.repeat(s, 32, axis=-1) / 2).all()


def test_scale_by_hand():
    """a = 7: s = 1.  a = 1: 1/7 = 0.14285.. = 18.28/128 -> 18/128.  a = 3.5 * 33 = 115.5 -> 16.5 is a tie
    between 16 and 17 (five bits): even, 16."""
    for a, want in ((7.0, 1.0), (1.0, 18 / 128), (115.5, 16.0), (122.5, 18.0), (0.0, 0.0), (2.0 ** -130, 0.0)):
        x = np.zeros(32)
        x[5] = -a
        codes, s = oracle.q4_round(x)
        assert s[0] == want
        assert codes[5] == (0 if want == 0 else -round(a / want))
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones(64)
        x[3] = bad
        codes, s = oracle.q4_round(x)
        assert s[0] == 0 and (codes[:32] == 0).all() and s[1] == 18 / 128 and (codes[32:] == 7).all()


@pytest.mark.parametrize("D", [64, 128])
def test_write_then_read(D):
    rng = np.random.default_rng(2)
    pool = np.full((3, 2, 18 * D), 0x5A, dtype=np.uint8)
    rows = {}
    for slot in (0, 15, 16, 37):
        for h in (0, 1):
            k, v = _bf16(rng, D), _bf16(rng, D)
            oracle.q4_write(pool, slot, h, k, False)
            oracle.q4_write(pool, slot, h, v, True)
            rows[slot, h] = k, v
    K, V = oracle.q4_read(pool, D)
    for (slot, h), (k, v) in rows.items():
        assert np.array_equal(K[slot // 16, h, slot % 16], oracle.q4_values(k))
        assert np.array_equal(V[slot // 16, h, slot % 16], oracle.q4_values(v))


def test_nibble_places_are_a_permutation():
    from oracle.q4 import nibble_index
    for D in (64, 128):
        for is_v in (False, True):
            assert sorted(nibble_index(D, d, is_v) for d in range(D)) == list(range(D))


def test_metadata_from_lengths_matches_the_scheduler():
    """The same rows through the packing oracle (which orders decodes before chunks) give the same metadata."""
    states = [(37, 0), (64, 0), (100, 0), (0, 12)]
    tables, nxt = [], 0
    for c, r in states:
        n = -(-(c + max(r, 1)) // 16)
        tables.append(np.arange(nxt, nxt + n, dtype=np.int32))
        nxt += n
    rows, _ = oracle.schedule(states, 8)
    ref = oracle.batch_metadata(rows, tables, 4, num_decodes=3)
    pad = np.full((4, 8), -1)
    for i, t in enumerate(tables):
        pad[i, :len(t)] = t
    got = oracle.metadata_from_lengths([37, 64, 100, 0], [1, 1, 1, 5], pad, 8)
    for k in ("cu_seqlens_q", "q_start_pos", "context_lens", "positions", "slot_mapping"):
        assert list(ref[k]) == got[k], k
    assert got["info"] == [8, 3 + 5 + 7 + 1, 3, 0]
    # the same step when each request holds only the pages of its cached tokens
    free = list(range(90, 100))
    got = oracle.metadata_from_lengths([37, 64, 100, 0], [1, 1, 1, 5], pad, 10, free=free, count=10)
    assert got["free_count"] == 8 and got["tables"][1, 4] == 99 and got["tables"][3, 0] == 98
    assert got["slot_mapping"][1] == 99 * 16 and got["slot_mapping"][3:8] == [98 * 16 + i for i in range(5)]
    assert got["positions"][8:] == [0, 0] and got["slot_mapping"][8:] == [-1, -1]


# ---------------------------------------------------------------------------- argument checks, no GPU needed

@pytest.fixture(scope="module")
def ms():
    from chunked_prefill_mixed_decode_gb300 import build
    build.build()
    import chunked_prefill_mixed_decode_gb300 as ms
    return ms


def test_block_bytes(ms):
    assert ms.q4_block_bytes(64) == 1152 and ms.q4_block_bytes(128) == 2304
    for D in (0, 32, 96, 256):
        with pytest.raises(ValueError):
            ms.q4_block_bytes(D)


def test_abi_refusals(ms):
    """Sizes and pointers that a call refuses before it launches anything (fake addresses, never read)."""
    lib, P = ms.lib(), 1 << 20

    def append(q=P, k=P, v=P, pos=P, slot=P, T=4, cos=P, sin=P, max_pos=64, kv=P, pages=4, q_rot=P, H_q=8, H_kv=2, D=128,
               page=16):
        return lib.ms_kv_append_rope_q4(q, k, v, pos, slot, T, cos, sin, max_pos, kv, pages, q_rot, H_q, H_kv, D, page,
                                        None, None)

    def read(kv=P, pages=4, slots=P, n=3, k=P, v=P, H=2, D=128, page=16):
        return lib.ms_kv_read_q4(kv, pages, slots, n, k, v, H, D, page, None, None)

    def attend(q=P, kv=P, pages=4, cu=P, qs=P, ctx=P, bt=P, off=None, bt_len=0, stride=4, rows=2, tokens=2, total=64, H_q=8,
               H_kv=2, D=128, page=16, scale=0.1, out=P, ws=P, ws_bytes=1 << 40):
        return lib.ms_mixed_step_attention_q4(q, kv, pages, cu, qs, ctx, bt, off, bt_len, stride, rows, tokens, total, H_q,
                                              H_kv, D, page, scale, out, ws, ws_bytes, None)

    for kw in (dict(T=-1), dict(D=96), dict(page=32), dict(H_q=7), dict(H_kv=0), dict(pages=-1), dict(max_pos=0), dict(q=0),
               dict(kv=0), dict(kv=P + 8), dict(slot=0), dict(q_rot=0), dict(cos=P + 4)):
        assert append(**kw) == ms.MS_ERR_ARG, kw
    assert append(T=0) == ms.MS_OK
    for kw in (dict(n=-1), dict(D=32), dict(H=0), dict(page=8), dict(kv=0), dict(k=P + 2), dict(v=0), dict(slots=0),
               dict(pages=-1)):
        assert read(**kw) == ms.MS_ERR_ARG, kw
    assert read(n=0) == ms.MS_OK
    for kw in (dict(rows=-1), dict(tokens=-1), dict(total=-1), dict(H_q=9), dict(H_q=6), dict(D=256), dict(page=8),
               dict(scale=0.0), dict(scale=float("nan")), dict(q=0), dict(kv=0), dict(kv=P + 8), dict(cu=0), dict(bt=0),
               dict(out=0), dict(ws=0), dict(ws=P + 16), dict(ws_bytes=64), dict(pages=0), dict(stride=0),
               dict(off=P, bt_len=0), dict(rows=8193), dict(tokens=(1 << 21) + 1)):
        assert attend(**kw) == ms.MS_ERR_ARG, kw
    assert attend(rows=0) == ms.MS_OK and attend(tokens=0) == ms.MS_OK

    def meta(c=P, d=P, R=2, tab=P, ts=4, free=None, fcap=0, fc=None, fs=None, pages=8, cap=16, cu=P, qs=P, ctx=P, pos=P,
             slot=P, bt=P, stride=4, off=None, btp=None, capp=0):
        return lib.ms_build_batch_metadata_device(c, d, R, tab, ts, free, fcap, fc, fs, pages, cap, cu, qs, ctx, pos, slot,
                                                  bt, stride, off, btp, capp, None, None, None)

    for kw in (dict(R=0), dict(R=8193), dict(ts=0), dict(cap=-1), dict(cap=(1 << 21) + 1), dict(pages=-1),
               dict(pages=(1 << 27) + 1), dict(c=0), dict(d=0), dict(tab=0), dict(cu=0), dict(qs=0), dict(ctx=0),
               dict(pos=0), dict(slot=0), dict(bt=0), dict(stride=0), dict(off=P), dict(off=P, btp=P, capp=4),
               dict(bt=0, off=P, capp=4), dict(free=P), dict(free=P, fc=P, fcap=4), dict(fc=P, fs=P), dict(btp=P),
               dict(free=P, fc=P, fs=P, fcap=-1)):
        assert meta(**kw) == ms.MS_ERR_ARG, kw


def test_metadata_refuses_overlapping_arrays(ms):
    """Inputs that an output would overwrite while other CTAs read them."""
    lib, R, ts, cap, fcap = ms.lib(), 5, 6, 40, 7
    at = {n: (i + 1) << 20 for i, n in enumerate("c d tab free fc fs cu qs ctx pos slot bt off btp info".split())}
    sizes = dict(c=R, d=R, tab=R * ts, free=fcap, fs=2, cu=R + 1, qs=R, ctx=R, pos=cap, slot=cap, bt=R * 8, off=R + 1, btp=30,
                 info=4)

    def meta(ragged, **kw):
        a = {**at, **kw}
        return lib.ms_build_batch_metadata_device(
            a["c"], a["d"], R, a["tab"], ts, a["free"], fcap, a["fc"], a["fs"], 50, cap, a["cu"], a["qs"], a["ctx"], a["pos"],
            a["slot"], None if ragged else a["bt"], 0 if ragged else 8, a["off"] if ragged else None,
            a["btp"] if ragged else None, 30 if ragged else 0, a["info"], None, None)

    for ragged in (False, True):
        for src in ("c", "d", "tab", "free"):
            for dst in ("cu", "qs", "ctx", "pos", "slot", "info") + (("off", "btp") if ragged else ("bt",)):
                for to in (at[src], at[src] + 4 * (sizes[src] - 1), at[src] - 4 * (sizes[dst] - 1)):  # alike, last, first word
                    assert meta(ragged, **{dst: to}) == ms.MS_ERR_ARG, (src, dst)
        assert meta(ragged, free=at["tab"] + 4) == ms.MS_ERR_ARG
        assert meta(ragged, fs=at["tab"]) == ms.MS_ERR_ARG and meta(ragged, fs=at["free"] - 4) == ms.MS_ERR_ARG


def test_binding_refusals(ms):
    torch = pytest.importorskip("torch")
    bf, i32 = torch.bfloat16, torch.int32
    q, k = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, 2, 64, dtype=bf)
    pos, tab = torch.zeros(3, dtype=i32), torch.zeros(8, 32)
    pool = torch.zeros(2, 2, 1152, dtype=torch.uint8)

    def refuse(match, fn, *a, **kw):
        with pytest.raises(ValueError, match=match):
            fn(*a, **kw)

    ap = ms.kv_append_rope_q4
    refuse("CUDA", ap, q, k, k, pos, pos, tab, tab, pool)
    refuse("kv_cache", ap, q, k, k, pos, pos, tab, tab, pool[..., :-1])
    refuse("kv_cache", ap, q, k, k, pos, pos, tab, tab, pool.to(torch.int8))
    refuse("kv_cache", ap, q, k, k, pos, pos, tab, tab, pool.view(4, 1152))
    refuse("k must have shape", ap, q, k[:2], k, pos, pos, tab, tab, pool)
    refuse("q must be", ap, q.float(), k, k, pos, pos, tab, tab, pool)
    refuse("contiguous", ap, q.transpose(0, 1), k, k, pos, pos, tab, tab, pool)
    refuse("slot_mapping", ap, q, k, k, pos, pos.long(), tab, tab, pool)
    rd = ms.kv_read_q4
    refuse("CUDA", rd, pool, pos, k, k)
    refuse("KV heads", rd, pool, pos, q, q)
    refuse("v_out", rd, pool, pos, k, k[:2])
    refuse("slots", rd, pool, pos[:2], k, k)
    at = ms.mixed_step_attention_q4
    cu, one, ws = torch.zeros(2, dtype=i32), torch.zeros(1, dtype=i32), torch.zeros(64, dtype=torch.uint8)
    bt = torch.zeros(1, 2, dtype=i32)
    refuse("CUDA", at, q, pool, cu, one, one, bt, 3, q, ws)
    refuse("kv_cache", at, q, pool.float(), cu, one, one, bt, 3, q, ws)
    refuse("out must have shape", at, q, pool, cu, one, one, bt, 3, q[:2], ws)
    refuse("context_lens", at, q, pool, cu, one, one[:0], bt, 3, q, ws)
    refuse("bt_offsets", at, q, pool, cu, one, one, bt, 3, q, ws, bt_offsets=one)
    md = ms.build_batch_metadata_device
    args = (one, one, bt, 4, cu, one, one, pos, pos)
    refuse("CUDA", md, *args, block_tables=bt)
    refuse("give block_tables", md, *args)
    refuse("give block_tables", md, *args, block_tables=bt, bt_offsets=cu, bt_pages=one)
    refuse("come together", md, *args, block_tables=bt, free_pages=one)
    refuse("free_state", md, *args, block_tables=bt, free_pages=one, free_count=one, free_state=one)
    refuse("slot_mapping", md, one, one, bt, 4, cu, one, one, pos, pos[:2], block_tables=bt)
    refuse("cu_seqlens_q", md, one, one, bt, 4, one, one, one, pos, pos, block_tables=bt)


def test_round_driver_refuses_graph_buckets_over_a_4_bit_pool(ms):
    torch = pytest.importorskip("torch")
    from chunked_prefill_mixed_decode_gb300.driver import RoundDriver
    pool = torch.zeros(4, 2, 1152, dtype=torch.uint8)
    with pytest.raises(ValueError, match="graph_buckets"):
        RoundDriver(ms.Engine(4, 8), pool, None, torch.zeros(8, 32), torch.zeros(8, 32), 4, 2, 64, graph_buckets=[8])


def test_metadata_refuses_overlapping_counts_and_status(ms):
    """The words of the free count and the status: written by one CTA while others read what lies under them."""
    lib, R, ts, cap, fcap = ms.lib(), 5, 6, 40, 7
    at = {n: (i + 1) << 20 for i, n in enumerate("c d tab free fc fs cu qs ctx pos slot bt off btp info st".split())}
    sizes = dict(c=R, d=R, tab=R * ts, free=fcap, fs=2, cu=R + 1, qs=R, ctx=R, pos=cap, slot=cap, bt=R * 8, off=R + 1, btp=30,
                 info=4, st=1)

    def meta(ragged, **kw):
        a = {**at, **kw}
        return lib.ms_build_batch_metadata_device(
            a["c"], a["d"], R, a["tab"], ts, a["free"], fcap, a["fc"], a["fs"], 50, cap, a["cu"], a["qs"], a["ctx"], a["pos"],
            a["slot"], None if ragged else a["bt"], 0 if ragged else 8, a["off"] if ragged else None,
            a["btp"] if ragged else None, 30 if ragged else 0, a["info"], a["st"], None)

    for ragged in (False, True):
        outs = ("cu", "qs", "ctx", "pos", "slot", "info") + (("off", "btp") if ragged else ("bt",))
        for src in ("c", "d", "tab", "free"):  # an input under the free state or the status word
            for to in (at[src], at[src] + 4 * (sizes[src] - 1)):
                assert meta(ragged, fs=to) == ms.MS_ERR_ARG and meta(ragged, st=to) == ms.MS_ERR_ARG, src
            assert meta(ragged, fs=at[src] - 4) == ms.MS_ERR_ARG, src
        for dst in outs + ("tab",):  # the free count, and the library's word, in an array that the call writes
            for to in (at[dst], at[dst] + 4 * (sizes[dst] - 1)):
                assert meta(ragged, fc=to) == ms.MS_ERR_ARG and meta(ragged, fs=to) == ms.MS_ERR_ARG, dst
        assert meta(ragged, fc=at["fs"] + 4) == ms.MS_ERR_ARG and meta(ragged, fc=at["st"]) == ms.MS_ERR_ARG
        assert meta(ragged, fs=at["st"]) == ms.MS_ERR_ARG and meta(ragged, fs=at["st"] - 4) == ms.MS_ERR_ARG


def test_workspace_sizes(ms):
    """Only the 4-bit query has the room for chunk items in parts: at D = 64 and G = 1 (256 rows of 264 bytes and 16 a
    part, 152 parts) 10.3 MB, at 128 20.2 MB, less for steps of few tokens and none for one token; the bf16 steps'
    own size is that of their layout."""
    def extra(*a):
        return ms.attention_workspace_size(*a) - ms.attention_workspace_size(*a, q4=False)
    assert 0 <= extra(7, 5000, 90000, 8, 8, 64) - 152 * (16 + 256 * 264) < 512
    assert 0 <= extra(7, 5000, 90000, 32, 8, 128) - 152 * (16 + 256 * 520) < 512
    assert 0 <= extra(7, 3, 90000, 32, 8, 128) - 152 * (16 + 12 * 520) < 512
    assert extra(7, 1, 90000, 32, 8, 128) < 256 and extra(0, 0, 0, 4, 4, 64) < 256
    assert ms.attention_workspace_size(1, 1, 0, 4, 2, 96) == 0 and ms.attention_workspace_size(1, 2, 0, 4, 3, 64) == 0
    # the layout of a 65-row step of 512 tokens over 262144 keys, 32 heads of 128: header, tables, items, and for each
    # of the 512 + 130 splits and heads a record of (max, sum) and 128 sums
    n = ms.attention_workspace_size(65, 512, 262144, 32, 32, 128, q4=False)
    records = 32 * (512 + 130) * (8 + 128 * 4)
    assert records < n < records + (1 << 20)
    # a replayed graph is one over bf16 pools
    import ctypes
    arr = (ctypes.c_int32 * 2)(8, 512)
    cfg = ms.GraphConfig(32, 32, 128, 16384, 65, 300, 4096, 0.1, 2, arr)
    assert n <= ms.lib().ms_graph_workspace_size(ctypes.byref(cfg)) < n + (1 << 20)


def test_batch_from_tables_has_no_host_copy(ms):
    """A batch built on the GPU copies no metadata: 0 bytes from the host; one from the host counts its arrays."""
    torch = pytest.importorskip("torch")
    from chunked_prefill_mixed_decode_gb300 import step
    tables = step.StepTables(torch.zeros(3, 4, dtype=torch.int32), 12, 8)
    assert tables.batch.h2d_bytes == 0 and not tables.batch.ragged
    meta = ms.build_batch_metadata([(5, 0), (0, 3)], [np.array([0]), np.array([1])], 8)
    assert step.to_device(meta, "cpu").h2d_bytes == 4 * (3 + 2 + 2 + 4 + 4 + 2)
