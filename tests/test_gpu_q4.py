"""The 4-bit cache on the GPU against plain 64-bit forms.

Bytes, whole numbers and q_rot are compared bit for bit.  Attention has a bound
from its arithmetic, per element: the output's rounding to bf16, half a step,
2^-8 |ref|; the rounding of each weight (a probability times V's scale) to bf16,
2^-8 of the sum A of p |v|; and 2^-10 A for everything in fp32.  The largest part
of that last term is the scores': a decode row's products carry code + 128, so a
score is off by at most about 2^-22 * 136 * sum |q| * s * scale, which for q ~
N(0, 1), s = 0.45 and D = 128 is 2e-4, and twice that for a probability.
"""
import numpy as np
import pytest

import oracle
import workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from chunked_prefill_mixed_decode_gb300 import build
    build.build()
    import chunked_prefill_mixed_decode_gb300 as ms
    from chunked_prefill_mixed_decode_gb300 import step
    return torch, ms, step


def _i32(torch, a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------- append and read

def _append(env, q, k, v, positions, slots, pool, max_pos):
    torch, ms, step = env
    H_q, D = q.shape[1:]
    cos, sin = step.rope_tables_device(max_pos, D, "cuda")
    q_rot = torch.full_like(q, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ms.kv_append_rope_q4(q, k, v, _i32(torch, positions), _i32(torch, slots), cos, sin, pool, q_rot=q_rot,
                         dev_status=status)
    return q_rot, ms.read_status(status)


def _oracle_append(q, k, v, positions, slots, pool, ok):
    """The oracle's bytes after the append of the tokens marked ok, and q_rot bits (or None) per token."""
    D = q.shape[-1]
    H_kv = k.shape[1]
    kb, vb, qb = (workloads.bf16_bits(x) for x in (k, v, q))
    cos, sin = oracle.rope_tables(np.maximum(positions, 0), D)
    kr, qr = oracle.rope_rotate(kb, cos, sin), oracle.rope_rotate(qb, cos, sin)
    out = pool.copy()
    for t, s in enumerate(slots):
        if ok[t]:
            for h in range(H_kv):
                oracle.q4_write(out, s, h, oracle.bf16_to_f64(kr[t, h]), False)
                oracle.q4_write(out, s, h, oracle.bf16_to_f64(vb[t, h]), True)
    return out, qr


@pytest.mark.parametrize("H_q,H_kv,D,T", [(4, 2, 64, 1), (8, 1, 128, 1), (8, 8, 128, 33), (40, 40, 64, 7),
                                          (32, 8, 128, 129), (3, 1, 64, 50), (16, 2, 64, 257)])
def test_append_bytes(env, H_q, H_kv, D, T):
    """Random slots over pages that other tokens share; what no token names keeps its bytes."""
    torch, ms, step = env
    rng = np.random.default_rng(T + D)
    g = torch.Generator(device="cuda").manual_seed(T)
    q, k, v = (torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16) for H in (H_q, H_kv, H_kv))
    pages = 2 + 2 * (-(-T // 16))
    before = rng.integers(0, 256, (pages, H_kv, 18 * D)).astype(np.uint8)
    pool = torch.from_numpy(before.copy()).cuda()
    slots = rng.permutation(16 * pages)[:T]
    positions = rng.integers(0, 5000, T)
    q_rot, status = _append(env, q, k, v, positions, slots, pool, 5000)
    assert status == 0
    want, qr = _oracle_append(q, k, v, positions, slots, before, [True] * T)
    np.testing.assert_array_equal(workloads.bf16_bits(q_rot), qr)
    np.testing.assert_array_equal(pool.cpu().numpy(), want)
    # and the same rows read back, twice each and in another order
    sl = np.concatenate([slots, slots[::-1]])
    ko, vo = (torch.empty(2 * T, H_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ms.kv_read_q4(pool, _i32(torch, sl), ko, vo)
    K, V = oracle.q4_read(want, D)
    np.testing.assert_array_equal(oracle.bf16_to_f64(workloads.bf16_bits(ko)), K[sl // 16, :, sl % 16])
    np.testing.assert_array_equal(oracle.bf16_to_f64(workloads.bf16_bits(vo)), V[sl // 16, :, sl % 16])


def test_append_values_at_the_edges(env):
    """Zeros, the smallest and the largest magnitudes, exact ties of the codes and of the scale, infinities and NaN."""
    torch, ms, step = env
    D = 128
    rows = [np.zeros(D), np.full(D, 2.0 ** -126), np.full(D, 2.0 ** -133), np.full(D, 3.3895313892515355e38),
            np.r_[7.0, np.arange(127) / 2 % 7], np.r_[115.5, np.full(127, 8.0)], np.r_[-122.5, np.full(127, 9.0)],
            np.r_[7 * 2.0 ** -126, np.full(127, 2.0 ** -127)], np.full(D, -2.0 ** -124)]
    bad = [np.r_[np.inf, np.ones(127)], np.r_[np.ones(40), np.nan, np.ones(87)], np.r_[np.ones(127), -np.inf]]
    x = torch.tensor(np.array(rows + bad), dtype=torch.float32, device="cuda").to(torch.bfloat16)[:, None]
    n = len(rows)
    for part, flag in ((x[:n], 0), (x[n:], ms.STATUS_NONFINITE)):
        part = part.contiguous()
        T = part.shape[0]
        pool = torch.full((1, 1, 18 * D), 0x33, dtype=torch.uint8, device="cuda")
        before = pool.cpu().numpy()
        _, status = _append(env, part, part, part, [0] * T, list(range(T)), pool, 1)  # position 0: no rotation
        assert status == flag
        want, _ = _oracle_append(part, part, part, np.zeros(T, int), range(T), before, [True] * T)
        np.testing.assert_array_equal(pool.cpu().numpy(), want)
    for r in range(len(bad)):  # one bad row at a time: whichever group holds it, it is reported
        one = x[n + r:n + r + 1].contiguous()
        pool = torch.zeros((1, 1, 18 * D), dtype=torch.uint8, device="cuda")
        ones = torch.ones_like(one)
        assert _append(env, ones, one, ones, [0], [0], pool, 1)[1] == ms.STATUS_NONFINITE
        assert _append(env, ones, ones, one, [0], [0], pool, 1)[1] == ms.STATUS_NONFINITE


def test_append_and_read_bad_slots_and_positions(env):
    torch, ms, step = env
    D, H_q, H_kv, pages = 64, 4, 2, 3
    q, k, v = (torch.randn(6, H, D, device="cuda").to(torch.bfloat16) for H in (H_q, H_kv, H_kv))
    for slots, positions, flag in (([0, -1, 47, 5, -1, 9], [1] * 6, 0), ([0, 48, 47, 5, 6, 9], [1] * 6, 1),
                                   ([0, -2, 47, 5, 6, 9], [1] * 6, 1), ([0, 1, 2, 3, 4, 5], [0, 9, 10, 3, -1, 2], 2),
                                   ([0, 1, 99, 3, 4, 5], [0, 9, 10, 3, 1, 2], 3)):
        pool = torch.full((pages, H_kv, 18 * D), 0x21, dtype=torch.uint8, device="cuda")
        before = pool.cpu().numpy()
        q_rot, status = _append(env, q, k, v, positions, slots, pool, 10)
        assert status == flag
        in_table = [0 <= p < 10 for p in positions]
        ok = [0 <= s < 16 * pages and i for s, i in zip(slots, in_table)]
        want, qr = _oracle_append(q, k, v, np.clip(positions, 0, 9), slots, before, ok)
        np.testing.assert_array_equal(pool.cpu().numpy(), want)
        got = workloads.bf16_bits(q_rot)
        for t in range(6):  # a token outside the table writes nothing at all
            np.testing.assert_array_equal(got[t], qr[t] if in_table[t] else np.full_like(got[t], 0x40E0))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ko, vo = (torch.ones(3, H_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ms.kv_read_q4(pool, _i32(torch, [-1, 4, -1]), ko, vo, dev_status=status)
    assert ms.read_status(status) == 0 and not ko[0].any() and not vo[2].any() and ko[1].any()
    for bad in (-2, 48, 2 ** 31 - 1, -2 ** 31):
        ms.kv_read_q4(pool, _i32(torch, [3, bad, 4]), ko, vo, dev_status=status)
        assert ms.read_status(status) == ms.STATUS_BAD_SLOT and not ko[1].any() and ko[2].any()
    empty = torch.empty(0, H_kv, D, dtype=torch.bfloat16, device="cuda")
    ms.kv_read_q4(pool, _i32(torch, [0]), empty, empty)


# ---------------------------------------------------------------------------- metadata from lengths

def _meta_case(rng, R, max_c, max_d, p_idle=0.1):
    c = rng.integers(0, max_c + 1, R)
    d = np.where(rng.random(R) < 0.6, 1, rng.integers(0, max_d + 1, R))
    d[rng.random(R) < p_idle] = 0
    return c, d


class Meta:
    """Buffers and one call of build_batch_metadata_device; outputs start at a value no call writes."""

    def __init__(self, env, c, d, stride, cap, ragged, alloc, bt_stride=None, cap_pages=None, num_pages=None, count=None,
                 seed=0, alias=False):
        self.torch, self.ms, _ = env
        torch = self.torch
        R = len(c)
        rng = np.random.default_rng(seed)
        held = -(-np.asarray(c, dtype=np.int64) // 16)
        need = np.where(np.asarray(d) > 0, -(-(np.asarray(c, dtype=np.int64) + d) // 16), 0)
        total = int(held.sum() + np.maximum(need - held, 0).sum())
        self.num_pages = total + 10 if num_pages is None else num_pages
        ids = rng.permutation(max(self.num_pages, total + 10))
        self.tab = np.full((R, stride), -7, dtype=np.int64)
        at = 0
        for s in range(R):
            n = min(stride, int(held[s] if alloc else max(held[s], need[s])))
            self.tab[s, :n] = ids[at:at + n]
            at += n
        self.free = ids[at:] if alloc else None
        self.count = (len(self.free) if count is None else count) if alloc else 0
        E = lambda *n: torch.full(n, -99, dtype=torch.int32, device="cuda")  # noqa: E731
        self.c, self.d = _i32(torch, c), _i32(torch, d)
        self.tables = _i32(torch, self.tab)
        self.out = {"cu_seqlens_q": E(R + 1), "q_start_pos": E(R), "context_lens": E(R), "positions": E(cap),
                    "slot_mapping": E(cap)}
        if ragged:
            self.out["bt_offsets"] = E(R + 1)
            self.out["bt_pages"] = E(max(int(need.sum()) if cap_pages is None else cap_pages, 1))
        else:
            self.out["block_tables"] = E(R, stride if bt_stride is None else bt_stride)
        self.kw = {}
        if alloc:
            self.state = torch.tensor([self.count, 0], dtype=torch.int32, device="cuda")
            fc = self.state[:1] if alias else torch.tensor([self.count], dtype=torch.int32, device="cuda")
            if not alias:
                self.state[0] = -5
            self.kw = dict(free_pages=_i32(torch, self.free), free_count=fc, free_state=self.state)
        self.info = E(4)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(self, stream=None):
        self.ms.build_batch_metadata_device(self.c, self.d, self.tables, self.num_pages, **self.out, info=self.info,
                                            dev_status=self.status, stream=stream, **self.kw)

    def check(self, flag=0):
        assert self.ms.read_status(self.status) == flag
        c, d = self.c.cpu().numpy(), self.d.cpu().numpy()
        cap = self.out["positions"].numel()
        ref = oracle.metadata_from_lengths(c, d, self.tab, cap, self.free, self.count)
        for k in ("cu_seqlens_q", "q_start_pos", "context_lens", "positions", "slot_mapping"):
            np.testing.assert_array_equal(self.out[k].cpu().numpy(), ref[k], err_msg=k)
        if "bt_offsets" in self.out:
            np.testing.assert_array_equal(self.out["bt_offsets"].cpu().numpy(), ref["bt_offsets"])
            n = len(ref["bt_pages"])
            np.testing.assert_array_equal(self.out["bt_pages"][:n].cpu().numpy(), ref["bt_pages"])
            assert (self.out["bt_pages"][n:] == -99).all()
        else:
            bt = self.out["block_tables"].cpu().numpy()
            for s in range(len(c)):
                row = ref["bt_pages"][ref["bt_offsets"][s]:ref["bt_offsets"][s + 1]]
                np.testing.assert_array_equal(bt[s], row + [-1] * (bt.shape[1] - len(row)))
        np.testing.assert_array_equal(self.tables.cpu().numpy(), ref["tables"])
        assert self.info.tolist() == ref["info"]
        if self.free is not None:
            assert self.state.tolist() == [ref["free_count"], 0]

    def check_refused(self, flag):
        """The step became one of pad rows; no page was taken."""
        assert self.ms.read_status(self.status) == flag
        for k in ("cu_seqlens_q", "q_start_pos", "context_lens", "positions", "bt_offsets"):
            assert k not in self.out or not self.out[k].any(), k
        assert (self.out["slot_mapping"] == -1).all()
        if "block_tables" in self.out:
            assert (self.out["block_tables"] == -1).all()
        else:
            assert (self.out["bt_pages"] == -99).all()
        np.testing.assert_array_equal(self.tables.cpu().numpy(), self.tab)
        assert self.info.tolist() == [0, 0, 0, 0]
        if self.free is not None:
            assert self.state.tolist() == [self.count, 0]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("alloc", [False, True])
@pytest.mark.parametrize("R,max_c,max_d", [(1, 40, 20), (3, 0, 5), (33, 300, 40), (511, 700, 3), (513, 64, 900),
                                           (8192, 100, 2)])
def test_metadata(env, R, max_c, max_d, alloc, ragged):
    rng = np.random.default_rng(R + max_c)
    c, d = _meta_case(rng, R, max_c, max_d)
    if R == 1:
        d[:] = max_d
    stride = -(-(max_c + max_d + 16) // 16)
    m = Meta(env, c, d, stride, int(d.sum()) + 13, ragged, alloc, seed=R, alias=R % 2 == 0)
    m.call()
    m.check()


def test_metadata_long_rows_and_exact_capacities(env):
    """Rows of 130000 tokens, a chunk of 9000, capacities with nothing to spare and a free list used up."""
    c, d = np.array([130000, 0, 131071, 16, 15]), np.array([1, 9000, 1, 1, 1])
    for ragged in (False, True):
        m = Meta(env, c, d, 8192, int(d.sum()), ragged, True, count=1 + 563 + 1, seed=5)
        m.free = m.free[:m.count]
        m.call()
        m.check()


def test_metadata_idle_rows_only(env):
    for alloc in (False, True):
        m = Meta(env, [100, 0, 7], [0, 0, 0], 8, 5, False, alloc)
        m.call()
        m.check()
        m = Meta(env, [100, 0, 7], [0, 0, 0], 8, 5, True, alloc, cap_pages=4)
        m.call()
        m.check()


def test_metadata_refusals_on_the_device(env):
    torch, ms, _ = env
    META, NOPG = ms.STATUS_BAD_META, ms.STATUS_NO_PAGES
    for ragged in (False, True):
        for c, d, kw, flag in (([5, -1], [1, 1], {}, META), ([5, 6], [1, -3], {}, META),
                               ([2 ** 31 - 1, 6], [1, 1], {}, META), ([5, 6], [9, 9], dict(cap=17), META),
                               ([5, 200], [1, 1], dict(stride=12, bt_stride=32), NOPG),
                               ([5, 2 ** 31 - 2], [1, 1], {}, META | NOPG),
                               ([16, 32, 48], [1, 1, 1], dict(alloc=True, count=2), NOPG),
                               ([16, 32, 48], [1, 1, 1], dict(alloc=True, count=-1), META | NOPG),
                               ([16, 32, 48], [1, 1, 1], dict(alloc=True, count=100000), META),
                               ([5, 40], [1, 1], dict(bt_stride=2, cap_pages=3), META)):
            small = [min(max(x, 0), 300) for x in c]
            m = Meta(env, small, d, kw.get("stride", 32), kw.get("cap", 24), ragged, kw.get("alloc", False),
                     bt_stride=kw.get("bt_stride"), cap_pages=kw.get("cap_pages", 30), count=kw.get("count"))
            if kw.get("alloc"):
                m.state[0] = m.count
            m.c = _i32(torch, c)
            m.call()
            m.check_refused(flag)


def test_metadata_bad_page_gets_no_slot(env):
    torch, ms, _ = env
    m = Meta(env, [20, 3, 40], [1, 14, 2], 4, 20, False, False)
    m.tables[1, 1] = m.num_pages
    m.call()
    assert ms.read_status(m.status) == ms.STATUS_BAD_PAGE
    slots = m.out["slot_mapping"].tolist()
    assert slots[14] == -1 and min(slots[:14]) >= 0 and min(slots[15:17]) >= 0


def test_metadata_replayed_as_the_lengths_grow(env):
    """One captured call replayed token by token: pages come from the free list as rows cross page ends."""
    torch, ms, _ = env
    c0, d = np.array([14, 31, 0, 47]), np.array([1, 1, 1, 0])
    m = Meta(env, c0, d, 8, 4, True, True, cap_pages=20, alias=True, seed=3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        m.call()
        m.c += m.d
    for n in range(40):
        m.out["bt_pages"].fill_(-99)
        graph.replay()
        torch.cuda.synchronize()
        m.c -= m.d  # check() reads the lengths that the call saw
        m.check()
        m.c += m.d
        m.tab, m.count = m.tables.cpu().numpy().astype(np.int64), int(m.state[0])


# ---------------------------------------------------------------------------- attention

def _pool(torch, pages, H_kv, D, seed, sigma=1.0):
    """A pool of rows that the append could have written (random codes -7..7, scales of five bits), and its values."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    NG = D // 32
    x = torch.randn(pages, H_kv, 2, 16 * D, generator=g, device="cuda") * 2.6 + 8
    nib = x.round().clamp(1, 15).to(torch.uint8)
    codes = nib[..., 0::2] | (nib[..., 1::2] << 4)
    s = torch.rand(pages, H_kv, 2, 16 * NG, generator=g, device="cuda") * 0.3 + 0.15
    u = (s * sigma).view(torch.int32) & ~0x7FFFF
    sc = u.view(torch.float32).to(torch.bfloat16).view(torch.uint8)
    return torch.cat([codes.reshape(pages, H_kv, -1), sc.reshape(pages, H_kv, -1)], -1).contiguous()


def _values(torch, pool, D):
    """K and V values [pages, H, 16, D] of a pool (fp64, GPU), by the oracle's nibble places."""
    from oracle.q4 import nibble_index
    out = []
    NG = D // 32
    for w in (0, 1):
        b = pool[..., w * 8 * D:(w + 1) * 8 * D].reshape(*pool.shape[:2], 16, D // 2)
        n = torch.tensor([nibble_index(D, d, w == 1) for d in range(D)], device="cuda")
        code = ((b[..., n // 2].int() >> (4 * (n % 2))) & 15).double() - 8
        sc = pool[..., 16 * D + w * 32 * NG:16 * D + (w + 1) * 32 * NG].contiguous().view(torch.bfloat16).double()
        out.append(code * sc.view(*pool.shape[:2], 16, NG).repeat_interleave(32, -1))
    return out


class Attn:
    def __init__(self, env, rows, H_q, H_kv, D, seed=0, ragged=False, sigma=1.0, qscale=1.0, slack_tokens=0, extra_stride=0,
                 pool=None):
        torch, ms, step = env
        self.torch, self.ms = torch, ms
        self.rows, self.H_q, self.H_kv, self.D, self.ragged = rows, H_q, H_kv, D, ragged
        rng = np.random.default_rng(seed)
        need = [-(-(c + d) // 16) for c, d in rows]
        total = max(sum(need), 1)
        self.pool = _pool(torch, total + 2, H_kv, D, seed, sigma) if pool is None else pool
        ids = rng.permutation(total + 2)
        self.pages, at = [], 0
        for n in need:
            self.pages.append(ids[at:at + n])
            at += n
        S = len(rows)
        stride = max(max(need), 1) + extra_stride
        bt = np.full((S, stride), -1)
        for s, pg in enumerate(self.pages):
            bt[s, :len(pg)] = pg
        cu = np.concatenate([[0], np.cumsum([d for _, d in rows])])
        self.T = int(cu[-1])
        self.bt = _i32(torch, bt)
        self.off = _i32(torch, np.concatenate([[0], np.cumsum(need)]))
        self.bt_pages = _i32(torch, np.concatenate(self.pages) if sum(need) else [0])
        self.cu, self.cun = _i32(torch, cu), cu
        self.start = _i32(torch, [c for c, _ in rows])
        self.ctx = _i32(torch, [c + d for c, d in rows])
        self.total = sum(c + d for c, d in rows)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        n = self.T + slack_tokens
        self.q = (torch.randn(n, H_q, D, generator=g, device="cuda") * qscale).to(torch.bfloat16)
        self.out = torch.full((n, H_q, D), 5.0, dtype=torch.bfloat16, device="cuda")
        w = ms.attention_workspace_size(S, n, self.total, H_q, H_kv, D)
        self.ws = torch.zeros(w, dtype=torch.uint8, device="cuda")

    def call(self, scale=None, stream=None, out=None, ws=None):
        self.ms.mixed_step_attention_q4(self.q, self.pool, self.cu, self.start, self.ctx,
                                        self.bt_pages if self.ragged else self.bt, self.total,
                                        self.out if out is None else out, self.ws if ws is None else ws,
                                        bt_offsets=self.off if self.ragged else None, scale=scale, stream=stream)

    def reference(self, scale=None):
        """Per token and head in 64 bits: softmax(scale q K) V, and the sum A of p |v|."""
        torch = self.torch
        scale = self.D ** -0.5 if scale is None else scale
        G = self.H_q // self.H_kv
        ref = torch.zeros(self.T, self.H_q, self.D, dtype=torch.float64, device="cuda")
        A = torch.zeros_like(ref)
        for s, (c, d) in enumerate(self.rows):
            if d == 0:
                continue
            pg = torch.tensor(np.asarray(self.pages[s]), device="cuda")
            K, V = (x.permute(1, 0, 2, 3).reshape(self.H_kv, -1, self.D)[:, :c + d]
                    for x in _values(torch, self.pool[pg], self.D))
            q = self.q[self.cun[s]:self.cun[s + 1]].double().view(d, self.H_kv, G, self.D).permute(1, 2, 0, 3)
            z = torch.einsum("hgtd,hnd->hgtn", q, K) * scale
            seen = torch.arange(c + d, device="cuda")[None] <= c + torch.arange(d, device="cuda")[:, None]
            p = torch.softmax(z.masked_fill(~seen, -float("inf")), -1)
            for dst, x in ((ref, V), (A, V.abs())):
                dst[self.cun[s]:self.cun[s + 1]] = torch.einsum("hgtn,hnd->thgd", p, x).reshape(d, self.H_q, self.D)
        return ref, A

    def check(self, scale=None, out=None):
        torch = self.torch
        assert self.ms.read_status(self.ws) == 0
        out = self.out if out is None else out
        ref, A = self.reference(scale)
        got = out[:self.T].double()
        assert torch.isfinite(got).all()
        err, bound = (got - ref).abs(), 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * A + 1e-30
        worst = (err / bound).max().item() if self.T else 0.0
        assert worst <= 1, worst
        assert (out[self.T:] == 5.0).all()
        return worst


SHAPES = [(4, 2, 64), (3, 3, 64), (8, 1, 64), (4, 1, 64), (2, 2, 128), (4, 2, 128), (8, 2, 128), (8, 1, 128), (16, 2, 128)]


@pytest.mark.parametrize("H_q,H_kv,D", SHAPES)
@pytest.mark.parametrize("ragged", [False, True])
def test_decode_rows(env, H_q, H_kv, D, ragged):
    """Contexts on both sides of every page and window end, from a single key to several thousand."""
    ctx = [0, 1, 14, 15, 16, 17, 30, 31, 32, 47, 63, 64, 65, 127, 255, 256, 511, 512, 513, 700, 1023, 2047, 4097, 6000]
    a = Attn(env, [(c, 1) for c in ctx], H_q, H_kv, D, seed=D + H_q, ragged=ragged)
    a.call()
    a.check()


@pytest.mark.parametrize("H_q,H_kv,D", SHAPES)
def test_chunk_rows(env, H_q, H_kv, D):
    """Chunks of 2 tokens up, at page-aligned and odd offsets, one alone longer than a pair of query tiles."""
    a = Attn(env, [(0, 2), (1, 3), (15, 2), (16, 16), (63, 65), (64, 64), (130, 33), (0, 300), (777, 129), (1000, 513)], H_q,
             H_kv, D, seed=D + H_q)
    a.call()
    a.check()


@pytest.mark.parametrize("H_q,H_kv,D", SHAPES)
@pytest.mark.parametrize("rows", [[(5000, 2)], [(9001, 40)], [(0, 700), (6000, 3)], [(3000, 200), (3100, 130), (20, 5), (1100, 64)],
                                  [(511, 2), (512, 2), (575, 65), (576, 129)], [(7990, 17), (4000, 1), (900, 1), (0, 0)],
                                  [(200 * i, 1) for i in range(40)] + [(12000, 33), (64, 64)]])
def test_few_chunk_rows(env, H_q, H_kv, D, rows):
    """Few items over long contexts: their keys are cut into parts, joined by the part that ends last.  Rows whose last
    part starts past their earlier tokens, rows too short to cut beside long ones, decodes beside them."""
    torch = env[0]
    a = Attn(env, rows, H_q, H_kv, D, seed=H_q + D + len(rows))
    a.call()
    a.check()
    first = a.out.clone()
    for cut in (0, 4096, 70000):  # less room for parts (80 KB at least with all of it); the same call again gives the same bits
        b = a.ws[:a.ws.numel() - cut]
        b.zero_()
        a.call(ws=b)
        if cut == 0:
            assert torch.equal(a.out, first)
        a.check()


@pytest.mark.parametrize("D", [64, 128])
def test_few_chunk_rows_ragged_and_replayed(env, D):
    """Parts over a ragged table, captured once and replayed as the rows' lengths change under it: cut, whole, cut."""
    torch, ms, _ = env
    H_q, H_kv = 8, 2
    big = Attn(env, [(9000, 30), (5000, 100), (700, 1)], H_q, H_kv, D, seed=70 + D, ragged=True, slack_tokens=2)
    big.call()
    big.check()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        big.call()
    first = big.out.clone()
    for rows in ([(9000, 30), (5000, 100), (700, 1)], [(40, 30), (60, 70), (0, 0)], [(8000, 129), (0, 1), (0, 2)]):
        rows_now = [(c, d) for c, d in rows]
        cu = np.concatenate([[0], np.cumsum([d for _, d in rows_now])])
        big.cu.copy_(_i32(torch, cu))
        big.start.copy_(_i32(torch, [c for c, _ in rows_now]))
        big.ctx.copy_(_i32(torch, [c + d for c, d in rows_now]))
        big.out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        assert rows_now != [(9000, 30), (5000, 100), (700, 1)] or torch.equal(big.out, first)
        a = Attn(env, rows_now, H_q, H_kv, D, pool=big.pool)
        a.pages = [pg[:-(-(c + d) // 16)] for pg, (c, d) in zip(big.pages, rows_now)]
        a.q, a.ws, a.out = big.q, big.ws, big.out
        a.check()


@pytest.mark.parametrize("H_q,H_kv,D,seed", [(8, 2, 128, 1), (4, 4, 64, 2), (8, 1, 64, 3), (32, 8, 128, 4)])
def test_mixed_rows_with_pads(env, H_q, H_kv, D, seed):
    """Decodes, chunks and rows without tokens, in any order; tokens that no row covers stay as they were."""
    rng = np.random.default_rng(seed)
    rows = []
    for _ in range(40):
        c = int(rng.integers(0, 3000))
        rows.append((c, int(rng.choice([0, 1, 1, 1, int(rng.integers(2, 150))]))))
    for ragged in (False, True):
        a = Attn(env, rows, H_q, H_kv, D, seed=seed, ragged=ragged, slack_tokens=9, extra_stride=3)
        a.call()
        a.check()


def test_many_rows(env):
    """8192 rows, and rows of one key."""
    rng = np.random.default_rng(9)
    a = Attn(env, [(int(c), 1) for c in rng.integers(0, 40, 8192)], 2, 1, 64, seed=9)
    a.call()
    a.check()


def test_long_decode_row(env):
    """One row of 131072 keys: many splits, joined at the end."""
    a = Attn(env, [(131071, 1), (3, 1)], 4, 1, 128, seed=10, ragged=True)
    a.call()
    a.check()


@pytest.mark.parametrize("qscale,sigma,scale", [(30.0, 1.0, None), (1.0, 1e-4, None), (1.0, 2.0 ** 14, 2.0 ** -18), (0.0, 1.0, None)])
def test_sharp_and_flat_scores(env, qscale, sigma, scale):
    """Scores in the hundreds, and all equal; cached values far below and above one."""
    for D in (64, 128):
        a = Attn(env, [(900, 1), (5, 1), (300, 140), (0, 20)], 8, 2, D, seed=11, qscale=qscale, sigma=sigma)
        a.call(scale=scale)
        if qscale > 1:  # the scores' own fp32 error grows with them: 2^-22 * 136 * sum |q| * s * scale
            assert a.ms.read_status(a.ws) == 0
            ref, A = a.reference(scale)
            e_s = 2 * 2.0 ** -22 * 136 * qscale * D * 0.8 * 0.45 * D ** -0.5
            bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10 + 2 * e_s) * A
            assert ((a.out.double() - ref).abs() <= bound).all()
        else:
            a.check(scale=scale)


@pytest.mark.parametrize("D", [64, 128])
def test_largest_scales(env, D):
    """Scales past 2^123, where 24 of them pass the largest bf16: read back exactly, and attended over."""
    torch, ms, _ = env
    rows = [(0, 2), (0, 3), (1, 2), (0, 1), (1, 1), (2, 1)]  # at most three keys: their sum stays below 2^128
    a = Attn(env, rows, 8, 2, D, seed=31, sigma=2.0 ** 125, qscale=2.0 ** -110)
    pages = a.pool.shape[0]
    sc = a.pool[..., 16 * D:].contiguous().view(torch.bfloat16)
    assert sc.max() > 2.0 ** 123.5 and sc.min() < 2.0 ** 123
    k, v = (torch.empty(16 * pages, 2, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ms.kv_read_q4(a.pool, _i32(torch, np.arange(16 * pages)), k, v)
    for got, want in zip((k, v), _values(torch, a.pool, D)):
        assert torch.equal(got.double(), want.permute(0, 2, 1, 3).reshape(got.shape))
    a.call(scale=2.0 ** -17)
    a.check(scale=2.0 ** -17)


def test_stale_bytes_past_the_context_are_not_read_as_values(env):
    """Every slot past a row's context holds code -8 and a NaN scale; so does every page of the pool that no row owns."""
    torch, ms, _ = env
    for D, H_q, H_kv in ((64, 4, 2), (128, 8, 2), (128, 2, 2)):
        a = Attn(env, [(0, 1), (16, 1), (37, 1), (600, 1), (100, 5), (200, 150), (3, 2)], H_q, H_kv, D, seed=12)
        ref_pool = a.pool.clone()
        NG = D // 32
        live = torch.zeros(a.pool.shape[0], 16, dtype=torch.bool, device="cuda")
        for s, (c, d) in enumerate(a.rows):
            for i, pg in enumerate(a.pages[s]):
                live[int(pg), :min(16, c + d - 16 * i)] = True
        p = a.pool
        for off, w in ((0, D // 2), (8 * D, D // 2)):
            v = p[..., off:off + 16 * w].reshape(*p.shape[:2], 16, w)
            v[~live[:, None].expand(-1, H_kv, -1)] = 0
            p[..., off:off + 16 * w] = v.reshape(*p.shape[:2], -1)
        for off in (16 * D, 16 * D + 32 * NG):
            v = p[..., off:off + 32 * NG].reshape(*p.shape[:2], 16, 2 * NG)
            v[~live[:, None].expand(-1, H_kv, -1)] = 0xFF
            p[..., off:off + 32 * NG] = v.reshape(*p.shape[:2], -1)
        a.call()
        got = a.out.clone()
        assert torch.isfinite(got.float()).all()
        a.pool = ref_pool
        a.check()


def test_bad_pages_and_bad_metadata(env):
    torch, ms, _ = env
    for bad in (-1, 10 ** 6):
        a = Attn(env, [(100, 1), (40, 1), (100, 30)], 4, 2, 128, seed=13)
        for s in (0, 2):
            a.bt[s, 2] = bad
        a.call()
        assert ms.read_status(a.ws) == ms.STATUS_BAD_PAGE
        ref, A = a.reference()
        assert ((a.out[1].double() - ref[1]).abs() <= 2.0 ** -7 * A[1] + 2.0 ** -7 * ref[1].abs()).all()
    for field, row, value in (("ctx", 0, 7), ("start", 1, -1), ("cu", 1, 5000), ("ctx", 2, 2 ** 31 - 1)):
        a = Attn(env, [(100, 1), (40, 1), (100, 30)], 4, 2, 64, seed=14)
        getattr(a, field)[row] = value
        a.call()
        assert ms.read_status(a.ws) == ms.STATUS_BAD_META
    # a good call on the same workspace afterwards
    b = Attn(env, [(100, 1), (40, 1), (100, 30)], 4, 2, 64, seed=14)
    b.ws = a.ws
    b.call()
    b.check()


def test_page_ids_past_32_bit_offsets(env):
    """A pool of more than 4 GB: the last pages' byte offsets do not fit in 32 bits."""
    torch, ms, _ = env
    D, H_kv = 128, 8
    pages = (1 << 32) // (H_kv * 18 * D) + 200
    pool = torch.zeros(pages, H_kv, 18 * D, dtype=torch.uint8, device="cuda")
    few = _pool(torch, 64, H_kv, D, 15)
    a = Attn(env, [(500, 1), (200, 90)], 32, H_kv, D, seed=15, pool=few)
    a.pages = [pg + pages - 64 for pg in a.pages]
    a.bt = torch.where(a.bt >= 0, a.bt + pages - 64, a.bt)
    pool[-64:] = few
    a.pool = pool
    a.call()
    a.check()
    # and the append and the read-back there
    slots = np.array([16 * pages - 1, 16 * pages - 37])
    q, k, v = (torch.randn(2, H, D, device="cuda").to(torch.bfloat16) for H in (8, 8, 8))
    _, status = _append(env, q, k, v, [3, 4], slots, pool, 8)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    ms.kv_read_q4(pool, _i32(torch, slots), ko, vo)
    assert status == 0
    np.testing.assert_array_equal(oracle.bf16_to_f64(workloads.bf16_bits(vo)),
                                  oracle.q4_values(oracle.bf16_to_f64(workloads.bf16_bits(v))))


def test_repeat_stream_and_replay_give_the_same_bits(env):
    """The same call again, on another stream, and captured and replayed, on workspaces of their own."""
    torch, ms, _ = env
    a = Attn(env, [(3000, 1), (64, 1), (500, 200), (8000, 1)], 8, 2, 128, seed=16)
    a.call()
    torch.cuda.synchronize()
    first = a.out.clone()
    a.check()
    side, ws2, out2 = torch.cuda.Stream(), torch.zeros_like(a.ws), torch.empty_like(a.out)
    side.wait_stream(torch.cuda.current_stream())
    a.call(stream=side, ws=ws2, out=out2)
    side.synchronize()
    assert torch.equal(out2, first)
    graph, ws3, out3 = torch.cuda.CUDAGraph(), torch.zeros_like(a.ws), torch.empty_like(a.out)
    with torch.cuda.graph(graph, stream=side):
        a.call(ws=ws3, out=out3)
    for _ in range(3):
        out3.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out3, first)


# ---------------------------------------------------------------------------- together

def test_decode_loop_captured_whole(env):
    """Metadata from lengths, append, attention: captured once, replayed for 40 tokens with no host data in between.
    Every step's cache bytes are the oracle's, and its outputs those of 64-bit attention over them."""
    torch, ms, step = env
    H_q, H_kv, D, R, pages, stride = 8, 2, 64, 5, 64, 12
    c0 = [0, 13, 16, 40, 0]
    new = [1, 1, 1, 1, 0]  # the last request is idle
    ids = list(range(pages))
    tab = np.full((R, stride), -1)
    for s, c in enumerate(c0):
        for j in range(-(-c // 16)):
            tab[s, j] = ids.pop(0)
    pool = _pool(torch, pages, H_kv, D, 17)
    ref_pool = pool.cpu().numpy().copy()
    c, d, tables = _i32(torch, c0), _i32(torch, new), _i32(torch, tab)
    E = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    cap = 8
    cu, start, ctx, positions, slots = E(R + 1), E(R), E(R), E(cap), E(cap)
    bt, info, status = E(R, stride), E(4), E(1)
    free = _i32(torch, ids)
    state = torch.tensor([len(ids), 0], dtype=torch.int32, device="cuda")
    cos, sin = step.rope_tables_device(16 * stride, D, "cuda")
    q, k, v = (torch.zeros(cap, H, D, dtype=torch.bfloat16, device="cuda") for H in (H_q, H_kv, H_kv))
    q_rot, out = torch.zeros_like(q), torch.zeros_like(q)
    ws = torch.zeros(ms.attention_workspace_size(R, cap, 16 * pages, H_q, H_kv, D), dtype=torch.uint8, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())

    def one_step():
        ms.build_batch_metadata_device(c, d, tables, pages, cu, start, ctx, positions, slots, block_tables=bt,
                                       free_pages=free, free_count=state[:1], free_state=state, info=info,
                                       dev_status=status)
        ms.kv_append_rope_q4(q, k, v, positions, slots, cos, sin, pool, q_rot=q_rot, dev_status=status)
        ms.mixed_step_attention_q4(q_rot, pool, cu, start, ctx, bt, 16 * pages, out, ws)
        c.add_(d)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        one_step()
    host_tab, host_c, count = tab.astype(np.int64), np.array(c0), len(ids)
    for n in range(40):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert ms.read_status(status) == 0 and ms.read_status(ws) == 0
        m = oracle.metadata_from_lengths(host_c, new, host_tab, cap, free=ids, count=count)
        host_tab, count = m["tables"], m["free_count"]
        np.testing.assert_array_equal(slots.tolist(), m["slot_mapping"])
        np.testing.assert_array_equal(tables.cpu().numpy(), host_tab)
        ok = [s >= 0 for s in m["slot_mapping"]]
        ref_pool, qr = _oracle_append(q, k, v, np.array(m["positions"]), m["slot_mapping"], ref_pool, ok)
        np.testing.assert_array_equal(workloads.bf16_bits(q_rot)[:4], qr[:4])
        np.testing.assert_array_equal(pool.cpu().numpy(), ref_pool)
        a = Attn(env, [(int(x), y) for x, y in zip(host_c, new)], H_q, H_kv, D, pool=pool, slack_tokens=4)
        a.pages = [host_tab[s, :-(-int(x + y) // 16)] if y else [] for s, (x, y) in enumerate(zip(host_c, new))]
        a.q, a.T, a.ws = q_rot, 4, ws
        a.out = torch.cat([out[:4], torch.full_like(out[:4], 5.0)])
        a.check()
        host_c = host_c + new
    assert state.tolist() == [count, 0] and c.tolist() == list(host_c)


def test_step_tables_and_run_step(env):
    """The same loop through StepTables and run_step_q4: a prompt enters in chunks while others decode, lengths and
    chunk sizes changing on the GPU under one captured step."""
    torch, ms, step = env
    H_q, H_kv, D, R, pages, stride, cap = 8, 1, 128, 3, 40, 12, 48
    pool = step.kv_pool_q4(pages, H_kv, D, "cuda")
    ref_pool = pool.cpu().numpy().copy()
    page_tables = torch.full((R, stride), -1, dtype=torch.int32, device="cuda")
    tables = step.StepTables(page_tables, pages, cap, free_pages=torch.arange(pages, dtype=torch.int32, device="cuda"))
    c, d = _i32(torch, [0] * R), _i32(torch, [0] * R)
    cos, sin = step.rope_tables_device(16 * stride, D, "cuda")
    q, k, v = (torch.zeros(cap, H, D, dtype=torch.bfloat16, device="cuda") for H in (H_q, H_kv, H_kv))
    q_rot, out = torch.zeros_like(q), torch.zeros_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = step.workspace_for(tables.batch, H_q, H_kv, D, "cuda")
    graph = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        b = tables.build(c, d)
        step.run_step_q4(q, k, v, b, cos, sin, pool, out, ws, q_rot=q_rot, dev_status=status)
        c.add_(d)
    host_c, host_tab, count = np.zeros(R, dtype=np.int64), np.full((R, stride), -1), pages
    for n, new in enumerate([(30, 0, 0), (1, 40, 0), (1, 7, 0), (1, 1, 5), (1, 1, 33), (0, 1, 1), (46, 1, 1), (1, 1, 1)]):
        d.copy_(_i32(torch, new))
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert ms.read_status(status) == 0 and ms.read_status(ws) == 0 and ms.read_status(tables.status) == 0
        m = oracle.metadata_from_lengths(host_c, new, host_tab, cap, free=list(range(pages)), count=count)
        host_tab, count = m["tables"], m["free_count"]
        np.testing.assert_array_equal(tables.slot_mapping.tolist(), m["slot_mapping"])
        assert tables.info.tolist() == m["info"]
        T = sum(new)
        ok = [s >= 0 for s in m["slot_mapping"]]
        ref_pool, _ = _oracle_append(q, k, v, np.array(m["positions"]), m["slot_mapping"], ref_pool, ok)
        np.testing.assert_array_equal(pool.cpu().numpy(), ref_pool)
        a = Attn(env, [(int(x) if y else 0, y) for x, y in zip(host_c, new)], H_q, H_kv, D, pool=pool)
        a.pages = [host_tab[s, :-(-int(x + y) // 16)] if y else [] for s, (x, y) in enumerate(zip(host_c, new))]
        a.q, a.ws, a.out = q_rot, ws, out[:T].clone()
        a.check()
        host_c = host_c + new
    assert int(tables.free_state[0]) == count


def test_attention_straight_after_the_tables(env):
    """No append between the metadata and the attention that reads it: requests that share all their pages but the last
    (contexts that sum to more than the pool), lengths changing under one captured pair of calls."""
    torch, ms, step = env
    H_q, H_kv, D, R, pages, stride, cap = 8, 2, 64, 40, 90, 50, 96
    pool = _pool(torch, pages, H_kv, D, 60)
    host_tab = np.array([np.r_[np.arange(stride - 1), stride - 1 + s] for s in range(R)])
    tables = step.StepTables(_i32(torch, host_tab), pages, cap, max_context=R * stride * 16)
    c, d = _i32(torch, [0] * R), _i32(torch, [0] * R)
    q = torch.randn(cap, H_q, D, device="cuda").to(torch.bfloat16)
    out = torch.zeros_like(q)
    ws = step.workspace_for(tables.batch, H_q, H_kv, D, "cuda")
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=st):
        b = tables.build(c, d)
        ms.mixed_step_attention_q4(q, pool, b.cu_seqlens_q, b.q_start_pos, b.context_lens, b.block_tables, b.context_total,
                                   out, ws)
    rng = np.random.default_rng(61)
    for n in range(12):
        new = np.where(rng.random(R) < 0.2, 0, 1)
        new[int(rng.integers(R))] = int(rng.integers(2, cap - R))
        cached = rng.integers(0, 16 * stride - cap, R)
        c.copy_(_i32(torch, cached))
        d.copy_(_i32(torch, new))
        graph.replay()
        torch.cuda.synchronize()
        assert ms.read_status(ws) == 0 and ms.read_status(tables.status) == 0
        a = Attn(env, [(int(x) if y else 0, int(y)) for x, y in zip(cached, new)], H_q, H_kv, D, pool=pool)
        a.pages = [host_tab[s, :-(-int(x + y) // 16)] if y else [] for s, (x, y) in enumerate(zip(cached, new))]
        a.q, a.ws, a.out = q, ws, out[:a.T].clone()
        a.check()


@pytest.mark.parametrize("H_q,H_kv,D,seed", [(4, 2, 64, 50), (8, 1, 128, 52)])
def test_engine_rounds_over_a_4_bit_pool(env, H_q, H_kv, D, seed):
    """Random arrivals through the engine and the round driver, pages freed and handed out again: the pool's bytes are
    the oracle's after every round, the outputs those of 64-bit attention over them."""
    torch, ms, step = env
    from chunked_prefill_mixed_decode_gb300.driver import RoundDriver
    pages = 40
    pool = step.kv_pool_q4(pages, H_kv, D, "cuda")
    ref_pool = pool.cpu().numpy().copy()
    cos, sin = step.rope_tables_device(pages * 16 + 1, D, "cuda")
    eng = ms.Engine(pages, 40, max_chunk_per_request=24)
    drv = RoundDriver(eng, pool, None, cos, sin, H_q, H_kv, D)
    rng = np.random.default_rng(seed)
    finished = 0
    for rnd in range(25):
        for _ in range(int(rng.integers(0, 3))):
            try:
                eng.add_request(int(rng.integers(1, 120)), int(rng.integers(2, 12)))
            except ms.MixedStepError:
                pass
        if eng.stats()["num_live"] == 0:
            continue
        q, k, v = (torch.randn(40, H, D, device="cuda").to(torch.bfloat16) for H in (H_q, H_kv, H_kv))
        rec = drv.step(q, k, v)
        m, T = rec["meta"], rec["meta"]["num_tokens"]
        ref_pool, qr = _oracle_append(q[:T], k[:T], v[:T], m["positions"], m["slot_mapping"], ref_pool, [True] * T)
        np.testing.assert_array_equal(pool.cpu().numpy(), ref_pool)
        np.testing.assert_array_equal(workloads.bf16_bits(drv.q_rot[:T]), qr)
        rows = [(int(c), int(n - c)) for c, n in zip(m["q_start_pos"], m["context_lens"])]
        a = Attn(env, rows, H_q, H_kv, D, pool=pool)
        a.pages = [m["block_tables"][s, :-(-(c + d) // 16)] for s, (c, d) in enumerate(rows)]
        a.q, a.ws, a.out = drv.q_rot[:T], drv.workspace, drv.out[:T].clone()
        a.check()
        finished += len(rec["finished"])
    assert finished >= 4


# ---------------------------------------------------------------------------- the metadata call's shared memory

_FRESH = """
import sys, threading
import torch
import chunked_prefill_mixed_decode_gb300 as ms

def one(R, rounds=1):
    i32 = lambda *n: torch.zeros(n, dtype=torch.int32, device="cuda")
    c, d, tab = i32(R) + 5, i32(R) + 1, torch.arange(R, dtype=torch.int32, device="cuda")[:, None].contiguous()
    cu, start, ctx, pos, slot, bt = i32(R + 1), i32(R), i32(R), i32(R), i32(R), i32(R, 1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    for _ in range(rounds):
        ms.build_batch_metadata_device(c, d, tab, R, cu, start, ctx, pos, slot, block_tables=bt, stream=stream)
    stream.synchronize()
    assert torch.equal(cu, torch.arange(R + 1, dtype=torch.int32, device="cuda")), R
    assert torch.equal(slot, 16 * tab[:, 0] + 5) and torch.equal(bt, tab), R

def threads(counts, rounds):
    failed = []
    def work(R):
        try:
            one(R, rounds)
        except BaseException as e:
            failed.append((R, repr(e)))
    ts = [threading.Thread(target=work, args=(R,)) for R in counts]
    [t.start() for t in ts]
    [t.join() for t in ts]
    assert not failed, failed

torch.zeros(1, device="cuda")
"""


@pytest.mark.parametrize("code", ["[one(R) for R in (3045, 3046, 3047, 3060, 3071, 3073, 8192)]", "one(3047)", "one(3071)",
                                  "threads((3100, 8192, 4000, 5000), 400)"])
def test_metadata_row_counts_in_a_fresh_process(env, code):
    """Row counts around the 48 KB of shared memory that a kernel has without asking, static arrays included, before any
    larger call of the process; and calls of different counts by several host threads at once."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FRESH + code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_read_of_no_row_is_bitwise_zero(env):
    """Slot -1 and slots outside the pool read as +0, whatever the outputs held."""
    torch, ms, _ = env
    for D in (64, 128):
        pool = _pool(torch, 2, 3, D, 80 + D)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        ko, vo = (torch.ones(5, 3, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        ms.kv_read_q4(pool, _i32(torch, [-1, 7, 32, -9, 31]), ko, vo, dev_status=status)
        assert ms.read_status(status) == ms.STATUS_BAD_SLOT
        for x in (ko, vo):
            bits = workloads.bf16_bits(x)
            assert not bits[[0, 2, 3]].any() and bits[[1, 4]].any()
        # and so do the rows of a pool of zeros
        ms.kv_read_q4(torch.zeros_like(pool), _i32(torch, [0, 7, 31, 16, -1]), ko, vo)
        assert not workloads.bf16_bits(ko).any() and not workloads.bf16_bits(vo).any()


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (4, 4, 64), (8, 1, 64)])
def test_largest_sums_of_values(env, H_q, H_kv, D):
    """Values just below the documented bound, keys * max |V| < 2^120, with weights that rise by 2^7.9 over the row, as
    far as they may before the reference maximum follows: every sum stays finite, whatever keys a warp or tile starts
    with.  4096 keys of |V| = 7 * 2^105: 2^119.8."""
    torch, ms, _ = env
    NG = D // 32
    for rows in ([(4095, 1)], [(4000, 96)], [(4095, 1), (3990, 100), (64, 1), (1000, 40)]):
        a = Attn(env, rows, H_q, H_kv, D, seed=90, pool=_pool(torch, 2 + sum(-(-(c + d) // 16) for c, d in rows), H_kv, D, 90))
        for pages in a.pages:
            for j, pg in enumerate(pages):
                blk = a.pool[int(pg)]
                blk[:, :8 * D] = 0x88 if j % 16 < 4 else 0xCC  # K: code 0 in the first 64 keys of every 256, else 4
                blk[:, 8 * D:16 * D] = 0xFF  # V: code 7, in every other head -7
                blk[1::2, 8 * D:16 * D] = 0x11
                sc = torch.tensor([0.125] * 16 * NG + [2.0 ** 105] * 16 * NG, device="cuda").to(torch.bfloat16)
                blk[:, 16 * D:] = sc.view(torch.uint8)
        a.q.fill_(1.0)
        scale = 7.9 * float(np.log(2)) / (0.5 * D)
        a.call(scale=scale)
        a.check(scale=scale)


def _score_slack(a, s, scale):
    """Bounds e[h, g, t, n] on the error of row s's scores, from each one's own products.

    A tensor-core product adds 16 exact terms to its fp32 accumulator, all 17 cut to 24 bits of the largest: 17 steps of
    2^-23 of the largest magnitude M among them.  Chunk rows: D / 16 such products of q with K (quarters of it, a factor
    that changes nothing).  Decode rows: two products a group, of q with 128 + nibble, one over the scales times -136
    sum q (in three bf16 parts, exact), a multiply-add a group.  Either kind: the factor scale * log2 e and the
    exponent's multiply-add, 2^-22 of the score.
    """
    torch, D, H_kv = a.torch, a.D, a.H_kv
    G, NG = a.H_q // H_kv, D // 32
    c, d = a.rows[s]
    n = c + d
    pool = a.pool[torch.tensor(np.asarray(a.pages[s]), device="cuda")]
    K = _values(torch, pool, D)[0].permute(1, 0, 2, 3).reshape(H_kv, -1, D)[:, :n]
    q = a.q[a.cun[s]:a.cun[s + 1]].double().view(d, H_kv, G, D).permute(1, 2, 0, 3)
    z = torch.einsum("hgtd,hnd->hgtn", q, K)
    unit = 17 * 2.0 ** -23

    def step_error(q_, k_):  # q [h, g, t, 16 m], k [h, n, 16 m]: m products in a row onto one accumulator
        e = acc = 0.0
        top = torch.maximum(q_.abs().amax(-1)[..., None] * k_.abs().amax(-1)[:, None, None], torch.zeros_like(z))
        for i in range(q_.shape[-1] // 16):
            acc = acc + torch.einsum("hgtd,hnd->hgtn", q_[..., 16 * i:16 * i + 16], k_[..., 16 * i:16 * i + 16])
            e = e + unit * torch.maximum(acc.abs(), top)
        return e

    if d > 1:
        e = step_error(q, K)
    else:
        sc = pool[..., 16 * D:16 * D + 32 * NG].contiguous().view(torch.bfloat16).double()
        sc = sc.view(*pool.shape[:2], 16, NG).permute(1, 0, 2, 3).reshape(H_kv, -1, NG)[:, :n]  # [h, n, group]
        # elements 0 to 3 of each quarter of a group go into its first product, 4 to 7 into its second
        order = [8 * t + i + 4 * half for half in (0, 1) for t in range(4) for i in range(4)]
        off = [-136.0 * q[..., 32 * g:32 * g + 32].sum(-1) for g in range(NG)]
        run = sum(off[g][..., None] * sc[:, None, None, :, g] for g in range(NG))
        biggest = torch.stack([off[g].abs()[..., None] * sc[:, None, None, :, g] for g in range(NG)]).amax(0)
        e = unit * torch.maximum(run.abs(), biggest)
        for g in range(NG):
            cols = [32 * g + i for i in order]
            nib = K[..., cols] / sc[..., g:g + 1] + 136.0
            s_g = sc[:, None, None, :, g]
            term = s_g * torch.einsum("hgtd,hnd->hgtn", q[..., cols], nib)
            run = run + term
            e = e + s_g * step_error(q[..., cols], nib) + 2.0 ** -24 * run.abs()
        assert (run - z).abs().max() <= 1e-9 * biggest.max()  # the same score
    return scale * (e + 2.0 ** -22 * z.abs())


@pytest.mark.parametrize("qscale", [4.0, 30.0])
@pytest.mark.parametrize("D", [64, 128])
def test_sharp_scores_row_by_row(env, D, qscale):
    """Scores up to the hundreds, each row within the bound that its own scores' errors e give: with eta = e^e - 1 a
    weight is off by a factor 1 +- eta, the output by (sum p eta |v| + |o| sum p eta) / (1 - sum p eta), and by the
    roundings of every test here."""
    torch, ms, _ = env
    rows = [(900, 1), (5, 1), (300, 140), (0, 20), (37, 1), (2000, 1), (1500, 3)]
    a = Attn(env, rows, 8, 2, D, seed=95 + D, qscale=qscale)
    a.call()
    assert ms.read_status(a.ws) == 0
    ref, A = a.reference()
    scale, G = D ** -0.5, 4
    for s, (c, d) in enumerate(rows):
        pg = torch.tensor(np.asarray(a.pages[s]), device="cuda")
        K, V = (x.permute(1, 0, 2, 3).reshape(2, -1, D)[:, :c + d] for x in _values(torch, a.pool[pg], D))
        q = a.q[a.cun[s]:a.cun[s + 1]].double().view(d, 2, G, D).permute(1, 2, 0, 3)
        z = torch.einsum("hgtd,hnd->hgtn", q, K) * scale
        seen = torch.arange(c + d, device="cuda")[None] <= c + torch.arange(d, device="cuda")[:, None]
        p = torch.softmax(z.masked_fill(~seen, -float("inf")), -1)
        w = p * torch.expm1(_score_slack(a, s, scale))
        X = w.sum(-1).permute(2, 0, 1).reshape(d, 8, 1)
        assert X.max() < (0.003 if d > 1 else 0.04)  # what the scores' errors can add is a few parts in a thousand, or hundred
        cut = slice(int(a.cun[s]), int(a.cun[s + 1]))
        o, sums = ref[cut].abs(), A[cut]
        e = (torch.einsum("hgtn,hnd->thgd", w, V.abs()).reshape(d, 8, D) + o * X) / (1 - X)
        # weights below 2^-126 of the largest are lost: 2001 of them at most, times |v| <= 8 * 0.45 * 2^-126, under 1e-30
        bound = 2.0 ** -8 * o + (2.0 ** -8 + 2.0 ** -10) * sums + 1.01 * e + 1e-30
        err = (a.out[cut].double() - ref[cut]).abs()
        assert (err <= bound).all(), (s, (err / bound).max())


@pytest.mark.parametrize("H_q,H_kv,D", [(4, 2, 64), (8, 1, 64), (2, 2, 128), (8, 2, 128), (8, 1, 128)])
def test_which_chunk_items_are_cut(env, H_q, H_kv, D):
    """Items of one pair of query tiles over 142 tiles of keys and more, alone and beside 40 decodes, run in parts
    (workspace header: word 12 the tiles to a part, word 6 the items); rows of 10 tiles and of many items run whole, and
    so does everything on a workspace without the room, with the same result within the bounds."""
    torch, ms, _ = env

    def plan(ws):
        return ws[:256].view(torch.int32)[[12, 6]].tolist()

    for rows, cut in (([(9001, 40 // (H_q // H_kv))], True), ([(200 * i, 1) for i in range(40)] + [(12000, 32 // (H_q // H_kv))], True),
                      ([(511, 2), (512, 2), (575, 65)], False), ([(5000, 1500)] * 12, False)):
        a = Attn(env, rows, H_q, H_kv, D, seed=100 + len(rows))
        a.call()
        tiles, items = plan(a.ws)
        a.check()
        if cut:
            n_kt = -(-(rows[-1][0] + rows[-1][1]) // 64)
            assert 8 <= tiles < n_kt and items == H_kv * -(-n_kt // tiles) and items > H_kv
        else:
            assert tiles == 0
        bare = torch.zeros(ms.attention_workspace_size(len(rows), a.T, a.total, H_q, H_kv, D, q4=False), dtype=torch.uint8,
                           device="cuda")
        a.out.fill_(5.0)
        a.call(ws=bare)
        assert plan(bare)[0] == 0 and ms.read_status(bare) == 0
        a.check()
        # 256 bytes more are less than one part needs
        a.call(ws=torch.cat([bare.zero_(), torch.zeros(256, dtype=torch.uint8, device="cuda")]))
        a.check()


def test_rotation_in_place(env):
    """The append and a whole step with q_rot left out: q holds the rotated values afterwards, bit for bit the others."""
    torch, ms, step = env
    for H_q, H_kv, D, T in ((8, 2, 128, 37), (4, 4, 64, 300), (3, 1, 64, 5)):
        g = torch.Generator(device="cuda").manual_seed(T)
        q, k, v = (torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16) for H in (H_q, H_kv, H_kv))
        pages = -(-T // 16)
        slots, positions = _i32(torch, np.arange(T)), _i32(torch, np.arange(T))
        cos, sin = step.rope_tables_device(T, D, "cuda")
        pools = [step.kv_pool_q4(pages, H_kv, D, "cuda") for _ in range(3)]
        q_rot = torch.empty_like(q)
        ms.kv_append_rope_q4(q, k, v, positions, slots, cos, sin, pools[0], q_rot=q_rot)
        mine = q.clone()
        ms.kv_append_rope_q4(mine, k, v, positions, slots, cos, sin, pools[1])
        assert torch.equal(mine, q_rot) and torch.equal(pools[1], pools[0])
        cu, start, ctx = _i32(torch, [0, T]), _i32(torch, [0]), _i32(torch, [T])
        b = step.DeviceBatch(cu, start, ctx, positions, slots, _i32(torch, [list(range(pages))]), 1, T, 0, T, {})
        ws = step.workspace_for(b, H_q, H_kv, D, "cuda", q4=True)
        out, want = torch.zeros_like(q), torch.zeros_like(q)
        if H_q // H_kv in (1, 2, 4, 8):
            mine = q.clone()
            assert step.run_step_q4(mine, k, v, b, cos, sin, pools[2], out, ws) is mine
            ms.mixed_step_attention_q4(q_rot, pools[0], cu, start, ctx, b.block_tables, T, want, ws)
            assert torch.equal(mine, q_rot) and torch.equal(pools[2], pools[0]) and torch.equal(out, want)
            assert ms.read_status(ws) == 0


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (4, 4, 64), (8, 1, 64)])
def test_stalled_copies_time_out_and_the_workspace_recovers(env, H_q, H_kv, D):
    """The kernel's waits made to run out (no work item published, no copy issued): the chunk phase's after 1 ms, the
    decode teams' after their 2 s; chunk rows whole and in parts, decode rows, both together.  The call ends, reports
    it, writes no output, and the next call on the workspace, with the tensor memory that the stalled one held, is
    right."""
    import time
    torch, ms, _ = env
    for rows in ([(5, 1), (600, 1), (9000, 1)], [(0, 300), (777, 129)], [(9001, 20)],
                 [(7 * i, 1) for i in range(100)] + [(100, 70), (64, 5)]):
        a = Attn(env, rows, H_q, H_kv, D, seed=110 + len(rows))
        for _ in range(1 if any(d == 1 for _, d in rows) else 2):
            a.out.fill_(5.0)
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            ms.test_attention_stall_q4(a.q, a.pool, a.cu, a.start, a.ctx, a.bt, a.total, a.out, a.ws, 1_000_000)
            torch.cuda.synchronize()
            assert time.perf_counter() - t0 < 10.0
            assert ms.read_status(a.ws) == ms.STATUS_TIMEOUT and (a.out == 5.0).all()
            a.call()
            a.check()
    for limit in (0, 99_999, 2_000_000_001):
        with pytest.raises(ms.MixedStepError):
            ms.test_attention_stall_q4(a.q, a.pool, a.cu, a.start, a.ctx, a.bt, a.total, a.out, a.ws, limit)


def test_pages_given_back_between_steps(env):
    """A pool of 12 pages serves six requests of 5 pages each in turn: a finished one's pages go behind the free ones, by
    operations on the GPU, and the next build hands them out again."""
    torch, ms, step = env
    R, pages, stride, cap = 2, 12, 6, 96
    tables = step.StepTables(torch.full((R, stride), -1, dtype=torch.int32, device="cuda"), pages, cap,
                             free_pages=torch.arange(pages, dtype=torch.int32, device="cuda"))
    c, d = _i32(torch, [0, 0]), _i32(torch, [0, 0])
    tab, free, count = np.full((R, stride), -1), list(range(pages)), pages
    hc = np.zeros(R, dtype=np.int64)
    for n in range(12):
        new = [72 if hc[s] == 0 else 1 for s in range(R)] if n else [72, 0]  # the second request starts a step later
        if n and sum(new) > cap:
            new[1] = 0
        d.copy_(_i32(torch, new))
        tables.build(c, d)
        m = oracle.metadata_from_lengths(hc, new, tab, cap, free=free, count=count)
        tab, count = m["tables"], m["free_count"]
        assert ms.read_status(tables.status) == 0
        np.testing.assert_array_equal(tables.slot_mapping.tolist(), m["slot_mapping"])
        np.testing.assert_array_equal(tables.page_tables.cpu().numpy(), tab)
        c += d
        hc = hc + new
        for s in range(R):
            if hc[s] >= 74:  # finished: its five pages back, and the row to the next request
                at = tables.free_state[0].long() + torch.arange(5, device="cuda")
                tables.free_pages.index_copy_(0, at, tables.page_tables[s, :5])
                tables.free_state[0] += 5
                tables.page_tables[s] = -1
                c[s] = 0
                free[count:count + 5], count, hc[s] = [int(x) for x in tab[s, :5]], count + 5, 0
                tab[s] = -1
    assert tables.free_state.tolist() == [count, 0] and tables.free_pages[:count].tolist() == free[:count]


def test_two_steps_at_once(env):
    """Two attention calls in flight on two streams, each with its workspace: the bits of each one alone."""
    torch, ms, _ = env
    a = Attn(env, [(3000, 1), (500, 200), (8000, 1)], 8, 2, 128, seed=120)
    b = Attn(env, [(9001, 20), (77, 1), (64, 300)], 4, 4, 64, seed=121)
    want = []
    for x in (a, b):
        x.call()
        x.check()
        want.append(x.out.clone())
        x.outs = [torch.empty_like(x.out) for _ in range(20)]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for i in range(20):
        for x, st in zip((a, b), streams):
            x.call(stream=st, out=x.outs[i])
    torch.cuda.synchronize()
    for x, w in zip((a, b), want):
        assert all(torch.equal(o, w) for o in x.outs) and ms.read_status(x.ws) == 0


def test_a_step_that_the_tables_refuse_computes_nothing(env):
    """The free list runs short: the step becomes one of pad rows, the append and the attention after it leave cache and
    output as they were, and the next step, with pages enough, is served."""
    torch, ms, step = env
    H_q, H_kv, D, pages, cap = 8, 2, 128, 3, 64
    pool = _pool(torch, pages, H_kv, D, 130)
    before = pool.clone()
    tables = step.StepTables(torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), pages, cap,
                             free_pages=torch.arange(pages, dtype=torch.int32, device="cuda"))
    cos, sin = step.rope_tables_device(64, D, "cuda")
    q, k, v = (torch.randn(cap, H, D, device="cuda").to(torch.bfloat16) for H in (H_q, H_kv, H_kv))
    q_rot, out = torch.empty_like(q), torch.full_like(q, 5.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = step.workspace_for(tables.batch, H_q, H_kv, D, "cuda", q4=True)
    c = _i32(torch, [0, 0])
    step.run_step_q4(q, k, v, tables.build(c, _i32(torch, [20, 17])), cos, sin, pool, out, ws, q_rot=q_rot, dev_status=status)
    assert ms.read_status(tables.status) == ms.STATUS_NO_PAGES and ms.read_status(status) == 0 and ms.read_status(ws) == 0
    assert torch.equal(pool, before) and (out == 5.0).all()
    assert tables.free_state.tolist() == [pages, 0] and (tables.page_tables == -1).all()
    step.run_step_q4(q, k, v, tables.build(c, _i32(torch, [20, 16])), cos, sin, pool, out, ws, q_rot=q_rot, dev_status=status)
    assert ms.read_status(tables.status) == 0 and ms.read_status(status) == 0 and ms.read_status(ws) == 0
    a = Attn(env, [(0, 20), (0, 16)], H_q, H_kv, D, pool=pool)
    a.pages = [[2, 1], [0]]
    a.q, a.ws, a.out = q_rot, ws, out
    a.check()
