"""Windowed attention with sinks, and cross attention, on the GPU against plain 64-bit forms.

The bound is the arithmetic's, per element: the output's rounding to bf16, half a step, 2^-8 |ref|; the rounding of each
weight to bf16, 2^-8 of the sum A of p |v|; and 2^-10 A for everything in fp32 (scores of magnitude up to a hundred,
whose products of 128 terms round to about 2^-24 * 100 * 12, twice that for a weight; the exponentials, 2^-22).
"""
import numpy as np
import pytest

import workloads
from oracle import rotary

pytestmark = pytest.mark.gpu

ALL = 2 ** 31 - 1
CH_TILES, CH_ITEMS = 12, 6  # words of the workspace header: KV tiles to a part, chunk items
SPLIT, KV_FORM = 7, 13  # pages to a decode split; how K and V of a page come to the chunk tiles (KvForm)


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


class Span:
    """rows: (c, d) of a windowed call, (keys, d) of a cross call (window None).  Cells that no token of their row sees hold
    infinities and NaN; table entries in front of a row's window hold page ids that no pool has."""

    def __init__(self, env, rows, H_q, H_kv, D, window, sinks=None, seed=0, ragged=False, qscale=1.0, slack=0, poison=True):
        torch, ms, _ = env
        self.torch, self.ms = torch, ms
        self.rows, self.H_q, self.H_kv, self.D, self.window, self.ragged = rows, H_q, H_kv, D, window, ragged
        self.cross = window is None
        rng = np.random.default_rng(seed)
        self.first = [0 if self.cross else max(0, c + 1 - window) for c, _ in rows]  # first key that any token of the row sees
        self.ends = [c if self.cross else c + d for c, d in rows]
        need = [-(-n // 16) for n in self.ends]
        gone = [f // 16 for f in self.first]
        held = sum(max(0, n - g) for n, g in zip(need, gone))
        ids, at = rng.permutation(held + 2), 0
        S, self.pages = len(rows), []
        bt = np.full((S, max(max(need), 1) + 1), -1)
        for s in range(S):
            n = max(0, need[s] - gone[s])
            self.pages.append(np.concatenate([rng.integers(held + 2, 2 ** 31, min(gone[s], need[s])), ids[at:at + n]]).astype(np.int64))
            at += n
            bt[s, :need[s]] = self.pages[s]
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.k, self.v = (torch.randn(held + 2, H_kv, 16, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        if poison:
            junk = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(torch.bfloat16)
            seen = torch.zeros(held + 2, 16, dtype=torch.bool)
            for s in range(S):
                j = np.arange(self.first[s], self.ends[s])
                seen[self.pages[s][j // 16], j % 16] = True
            hidden = (~seen).cuda()[:, None, :, None].expand(self.k.shape)
            for x in (self.k, self.v):
                x[hidden] = junk[torch.arange(int(hidden.sum()), device="cuda") % 3]
        cu = np.concatenate([[0], np.cumsum([d for _, d in rows])])
        self.T, self.cun = int(cu[-1]), cu
        self.bt, self.cu = _i32(torch, bt), _i32(torch, cu)
        self.off = _i32(torch, np.concatenate([[0], np.cumsum(need)]))
        self.bt_pages = _i32(torch, np.concatenate(self.pages) if sum(need) else [0])
        self.start, self.lens = _i32(torch, [c for c, _ in rows]), _i32(torch, self.ends)
        self.total = sum(self.ends)
        n = self.T + slack
        self.q = (torch.randn(n, H_q, D, generator=g, device="cuda") * qscale).to(torch.bfloat16)
        self.sinks = None
        if sinks is not None:
            self.sinks = torch.randn(H_q, generator=g, device="cuda") * sinks if isinstance(sinks, float) else torch.tensor(sinks, device="cuda")
        self.out = torch.full((n, H_q, D), 5.0, dtype=torch.bfloat16, device="cuda")
        self.ws = torch.zeros(ms.attention_workspace_size(S, n, self.total, H_q, H_kv, D), dtype=torch.uint8, device="cuda")

    def call(self, scale=None, stream=None, out=None, ws=None):
        out, ws = self.out if out is None else out, self.ws if ws is None else ws
        table, off = (self.bt_pages, self.off) if self.ragged else (self.bt, None)
        if self.cross:
            self.ms.mixed_step_cross_attention(self.q, self.k, self.v, self.cu, self.lens, table, self.total, out, ws,
                                               bt_offsets=off, scale=scale, stream=stream)
        else:
            self.ms.mixed_step_attention_window(self.q, self.k, self.v, self.cu, self.start, self.lens, table, self.total, out,
                                                ws, self.window, sinks=self.sinks, bt_offsets=off, scale=scale, stream=stream)

    def reference(self, scale=None):
        """Per token and head in 64 bits, and the sum A of p |v|."""
        torch = self.torch
        scale = self.D ** -0.5 if scale is None else scale
        G = self.H_q // self.H_kv
        ref = torch.zeros(self.T, self.H_q, self.D, dtype=torch.float64, device="cuda")
        A = torch.zeros_like(ref)
        for s, (c, d) in enumerate(self.rows):
            f, n = self.first[s], self.ends[s]
            if d == 0 or n == 0:
                continue
            j = np.arange(f, n)
            pg, at = torch.tensor(self.pages[s][j // 16], device="cuda"), torch.tensor(j % 16, device="cuda")
            K, V = (x[pg, :, at].double().transpose(0, 1) for x in (self.k, self.v))
            q = self.q[self.cun[s]:self.cun[s + 1]].double().view(d, self.H_kv, G, self.D).permute(1, 2, 0, 3)
            z = torch.einsum("hgtd,hnd->hgtn", q, K) * scale
            if not self.cross:
                jj, p = torch.arange(f, n, device="cuda")[None], c + torch.arange(d, device="cuda")[:, None]
                z = z.masked_fill((jj > p) | (jj <= p - self.window), -float("inf"))
            if self.sinks is not None:
                z = torch.cat([z, self.sinks.double().view(self.H_kv, G, 1, 1).expand(-1, -1, d, 1)], -1)
            p = torch.softmax(z, -1)[..., :n - f]
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
        worst = ((got - ref).abs() / (2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -10) * A + 1e-30)).max().item() if self.T else 0.0
        assert worst <= 1, worst
        assert (out[self.T:] == 5.0).all()
        for s in range(len(self.rows)):
            if self.ends[s] == 0:
                assert (out[self.cun[s]:self.cun[s + 1]] == 0).all()
        return worst

    def word(self, i):
        return int(self.ws[:256].view(self.torch.int32)[i])


SHAPES = [(4, 2, 64), (3, 3, 64), (8, 1, 64), (4, 1, 64), (2, 2, 128), (4, 2, 128), (8, 2, 128), (8, 1, 128), (16, 2, 128)]
CTX = [0, 1, 14, 15, 16, 17, 30, 31, 32, 47, 63, 64, 65, 127, 255, 256, 511, 512, 513, 700, 1023, 2047, 4097, 9000]
CHUNKS = [(0, 2), (1, 3), (15, 2), (16, 16), (63, 65), (64, 64), (130, 33), (0, 300), (777, 129), (1000, 513)]


@pytest.mark.parametrize("H_q,H_kv,D", SHAPES)
@pytest.mark.parametrize("window,sinks,ragged", [(1, None, False), (16, 2.0, True), (17, None, True), (100, 2.0, False),
                                                 (1500, 1.0, True), (ALL, None, False), (ALL, 3.0, True)])
def test_window_decode_rows(env, H_q, H_kv, D, window, sinks, ragged):
    """Contexts on both sides of every page's and window's end, from a single key to several splits."""
    a = Span(env, [(c, 1) for c in CTX], H_q, H_kv, D, window, sinks, seed=D + H_q, ragged=ragged)
    a.call()
    a.check()


@pytest.mark.parametrize("H_q,H_kv,D", [x for x in SHAPES if x[0] <= 4 * x[1]])
@pytest.mark.parametrize("window,sinks", [(16, 2.0), (100, None), (1500, 1.0), (ALL, None), (None, None)])
def test_decode_weights_keep_what_rounding_leaves(env, H_q, H_kv, D, window, sinks):
    """Up to 4 heads to a KV head a decode row's weights are two bf16 numbers, off by 2^-8 of 2^-8 at most: of the bound's
    rounding of the weights 2^-16 A is left, and what is in fp32 and the output's half step stay."""
    a = Span(env, [(c + (window is None), 1) for c in CTX], H_q, H_kv, D, window, sinks, seed=3 * D + H_q)
    a.call()
    a.check()
    ref, A = a.reference()
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -16 + 2.0 ** -10) * A + 1e-30
    assert ((a.out.double() - ref).abs() / bound).max().item() <= 1


@pytest.mark.parametrize("H_q,H_kv,D", [x for x in SHAPES if x[0] == 8 * x[1]])
@pytest.mark.parametrize("window,sinks", [(16, 2.0), (100, None), (1500, 1.0), (ALL, None), (None, None)])
def test_decode_weights_of_8_heads_keep_what_rounding_leaves(env, H_q, H_kv, D, window, sinks):
    """The same bound with 8 heads to a KV head, whose remainders take a product of their own."""
    a = Span(env, [(c + (window is None), 1) for c in CTX], H_q, H_kv, D, window, sinks, seed=3 * D + H_q)
    a.call()
    a.check()
    ref, A = a.reference()
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -16 + 2.0 ** -10) * A + 1e-30
    assert ((a.out.double() - ref).abs() / bound).max().item() <= 1


@pytest.mark.parametrize("H_q,H_kv,D", SHAPES)
@pytest.mark.parametrize("window,sinks,ragged", [(1, 2.0, False), (7, None, True), (64, None, False), (129, 2.0, True),
                                                 (400, None, False), (ALL, 1.0, False)])
def test_window_chunk_rows(env, H_q, H_kv, D, window, sinks, ragged):
    """Chunks of 2 tokens up, at page-aligned and odd offsets, windows shorter than a tile and longer than a chunk."""
    a = Span(env, CHUNKS, H_q, H_kv, D, window, sinks, seed=D + H_q, ragged=ragged)
    a.call()
    a.check()


@pytest.mark.parametrize("H_q,H_kv,D", SHAPES)
@pytest.mark.parametrize("rows,window", [([(9001, 40)], 9000), ([(9001, 40)], 3000), ([(20000, 2)], ALL), ([(0, 700), (6000, 3)], 2500),
                                         ([(3000, 200), (3100, 130), (20, 5), (1100, 64)], ALL), ([(7990, 17), (4000, 1), (900, 1), (0, 0)], 5000),
                                         ([(200 * i, 1) for i in range(40)] + [(12000, 33), (64, 64)], 4000)])
@pytest.mark.parametrize("sinks", [None, 2.0])
def test_window_few_chunk_rows(env, H_q, H_kv, D, rows, window, sinks):
    """Few items over long spans are cut into parts; without the room for them the same step runs whole."""
    torch, ms, _ = env
    a = Span(env, rows, H_q, H_kv, D, window, sinks, seed=H_q + D + len(rows))
    a.call()
    a.check()
    first = a.out.clone()
    small = ms.attention_workspace_size(len(rows), a.q.shape[0], a.total, H_q, H_kv, D, q4=False)
    for n in (a.ws.numel(), a.ws.numel() - 70000, small):
        b = a.ws[:n]
        b.zero_()
        a.call(ws=b)
        if n == a.ws.numel():
            assert torch.equal(a.out, first)  # the same call again: the same bits
        if n == small:
            assert a.word(CH_TILES) == 0
        a.check()


@pytest.mark.parametrize("rows,H_q,H_kv,D,window", [([(1023, 1)], 32, 8, 128, 1024), ([(1500, 1)], 20, 20, 64, None), ([(1999, 1)] * 20, 8, 8, 64, ALL),
                                                    ([(4095, 1)], 8, 1, 128, ALL)])
def test_few_decode_rows_get_the_splits_that_the_bound_has_places_for(env, rows, H_q, H_kv, D, window):
    """A bound above the contexts' sum, with the workspace for it, leaves room for more splits; the rows stay what they are."""
    torch, ms, _ = env
    a = Span(env, rows, H_q, H_kv, D, window, None if window is None else 1.0, seed=14)
    a.call()
    a.check()
    split, total = a.word(SPLIT), a.total
    pages = -(-max(a.ends) // 16)
    assert -(-pages // split) <= total // 512 + 1 + 2 * len(rows)  # a split needs a place: one per 32 pages, two a row
    a.total = total + 200000
    ws = torch.zeros(ms.attention_workspace_size(len(rows), a.T, a.total, H_q, H_kv, D), dtype=torch.uint8, device="cuda")
    a.out.fill_(5.0)
    a.call(ws=ws)
    a.total = total
    assert int(ws[:256].view(torch.int32)[SPLIT]) < split and ms.read_status(ws) == 0
    a.check()


def test_some_of_the_few_rows_were_cut(env):
    for H_q, H_kv, D in SHAPES:
        for window in (9000, None):
            a = Span(env, [(9001, 40)], H_q, H_kv, D, window)
            a.call()
            assert a.word(CH_TILES) > 0 and a.word(CH_ITEMS) > H_kv
            a.check()


@pytest.mark.parametrize("H_q,H_kv,D", SHAPES)
@pytest.mark.parametrize("ragged", [False, True])
def test_cross_rows(env, H_q, H_kv, D, ragged):
    """One token and many over 0, 1, .. keys; rows of no token; a prompt of several pairs of Q tiles over a short encoder."""
    rows = [(0, 1), (1, 1), (15, 1), (16, 1), (17, 1), (1500, 1), (6000, 1), (33, 0), (0, 0), (0, 5), (0, 300), (1, 2), (16, 16), (63, 3),
            (64, 130), (65, 64), (300, 700), (1, 513), (1500, 33), (0, 1)]
    a = Span(env, rows, H_q, H_kv, D, None, seed=D + H_q, ragged=ragged, slack=3)
    a.call()
    a.check()


@pytest.mark.parametrize("H_q,H_kv,D", SHAPES)
@pytest.mark.parametrize("rows", [[(12000, 4)], [(9001, 40), (0, 7)], [(6000, 300)], [(30000, 2), (16, 1), (0, 1), (500, 20)], [(0, 9)], [(0, 1)],
                                  [(64 * 16, 2)], [(1, 1)]])
def test_cross_few_rows(env, H_q, H_kv, D, rows):
    torch, ms, _ = env
    a = Span(env, rows, H_q, H_kv, D, None, seed=H_q)
    a.call()
    a.check()
    first = a.out.clone()
    a.out.fill_(5.0)
    a.call()
    assert torch.equal(a.out, first)
    b = a.ws[:ms.attention_workspace_size(len(rows), a.T, a.total, H_q, H_kv, D, q4=False)]
    a.call(ws=b)
    a.check()


@pytest.mark.parametrize("n", [31, 32, 33, 64, 600, 3000, 8192])
@pytest.mark.parametrize("window", [37, None])
def test_many_rows(env, n, window):
    """Around the row counts at which the prologue changes its form; pad rows, chunks and rows without keys among them."""
    rng = np.random.default_rng(n)
    rows = [(int(rng.integers(0, 200)), int(rng.choice([0, 1, 1, 1, 1, 2, 9]))) for _ in range(n)]
    a = Span(env, rows, 4, 2, 64, window, 1.0 if window else None, seed=n, slack=5)
    a.call()
    a.check()


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (4, 4, 64), (8, 1, 128)])
def test_window_of_everything_is_the_causal_call(env, H_q, H_kv, D):
    """Chunk rows run the same tiles in the same order: the causal call's bits, where no item is cut.  (Decode rows are
    split by a rule of their own: both are within the bound.)"""
    torch, ms, _ = env
    a = Span(env, CHUNKS, H_q, H_kv, D, ALL, seed=4)
    b = Span(env, [(c, 1) for c in CTX] + CHUNKS, H_q, H_kv, D, ALL, seed=4)
    for x in (a, b):
        ws = x.ws[:ms.attention_workspace_size(len(x.rows), x.T, x.total, H_q, H_kv, D, q4=False)]
        x.call(ws=ws)
        x.check()
        want = torch.empty_like(x.out)
        ws.zero_()
        ms.mixed_step_attention(x.q, x.k, x.v, x.cu, x.start, x.lens, x.bt, x.total, want, ws)
        x.check(out=want)
        if x is a:
            assert torch.equal(x.out, want)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("qscale,scale", [(30.0, None), (0.0, None), (1.0, 1e-6)])
def test_sharp_and_flat_scores(env, D, qscale, scale):
    a = Span(env, [(c, 1) for c in (0, 5, 700, 3000)] + [(100, 40), (2000, 130)], 8, 2, D, 513, 2.0, qscale=qscale, seed=7)
    a.call(scale)
    # scores up to some hundreds: their products round to 2^-24 * 500 * 4
    a.check(scale)


def test_sinks_at_the_ends_of_their_range(env):
    """-infinity is no sink; far below every score it weighs nothing, far above it takes everything; each head its own."""
    torch = env[0]
    rows, inf = [(0, 1), (15, 1), (3000, 1), (0, 40), (700, 129), (9000, 30)], float("inf")
    for window in (64, 2000, ALL):
        none = Span(env, rows, 8, 2, 64, window, None, seed=3)
        none.call()
        none.check()
        for value in (-inf, -3e38, -300.0):
            a = Span(env, rows, 8, 2, 64, window, [value] * 8, seed=3)
            a.call()
            a.check()
            if value == -inf:
                assert (a.out.float() - none.out.float()).abs().max() <= 2.0 ** -7
        a = Span(env, rows, 8, 2, 64, window, [300.0] * 8, seed=3)
        a.call()
        assert torch.isfinite(a.out).all() and a.out.float().abs().max() < 1e-30
        a = Span(env, rows, 8, 2, 64, window, [-inf, 0.0, 5.0, -5.0, 10.0, 300.0, -300.0, 1.0], seed=3)
        a.call()
        a.check()


def test_finite_sinks_beyond_what_their_logarithm_to_base_2_holds(env):
    """A finite sink takes part as it is up to the type's end, where times log2 e it would be infinite, in whole rows and in
    rows that are cut: a decode row in splits, a chunk row in parts, with the room for them and without.  Beside such a
    sink every weight is zero in 64 bits, and so is the row; heads with other sinks are those of the plain form."""
    torch, ms, _ = env
    top = float(torch.finfo(torch.float32).max)
    for H_q, H_kv, D in ((8, 2, 64), (8, 1, 128)):
        for rows, window in (([(9001, 1), (9001, 40)], ALL), ([(9001, 1), (9001, 40)], 5000), ([(40, 1), (90, 30)], 64)):
            a = Span(env, rows, H_q, H_kv, D, window, [3e38, top, 2.4e38, 0.0, -top, 2.3e38, 2.0, top], seed=8)
            a.call()
            if window > 64:
                assert a.word(SPLIT) < min(window, 9002) // 16 and a.word(CH_TILES) > 0
            a.check()
            assert (a.out[:, [0, 1, 2, 5, 7]] == 0).all()
            whole = torch.zeros(ms.attention_workspace_size(len(rows), a.T, a.total, H_q, H_kv, D, q4=False), dtype=torch.uint8,
                                device="cuda")
            a.out.fill_(5.0)
            a.call(ws=whole)
            a.check()


def test_sink_above_all_scores_and_then_keys_far_above_it(env):
    """The reference maximum starts at the sink and is raised by a later tile or split."""
    torch = env[0]
    for sink in (20.0, -20.0):
        a = Span(env, [(5000, 1), (300, 1), (400, 200), (6000, 50)], 4, 2, 64, ALL, [sink] * 4, seed=5, poison=False)
        for pg in a.pages:  # keys grow with their place in the row's pages
            for i, p in enumerate(pg):
                a.k[int(p)] *= 0.05 + 3.0 * i / len(pg)
        a.call()
        a.check()


def test_bad_pages_and_bad_metadata(env):
    torch, ms, _ = env
    for window in (100, None):
        rows = [(500, 1), (300, 40), (40, 1)]
        a = Span(env, rows, 8, 2, 64, window, poison=False)
        page = 18 if window is None else 31
        keep = int(a.bt[0, page])
        a.bt[0, page] = 10 ** 6
        a.call()
        assert ms.read_status(a.ws) == ms.STATUS_BAD_PAGE and torch.isfinite(a.out).all()
        a.bt[0, page] = keep
        for name, bad in (("lens", [500 if window else -1, 340, 41]), ("start", [500, -1, 40]), ("lens", [10 ** 6, 340, 41]),
                          ("cu", [0, 1, 0, 42]), ("cu", [0, 1, 41, 43])):
            if window is None and name == "start":
                continue
            old = getattr(a, name)
            setattr(a, name, _i32(torch, bad))
            a.out.fill_(5.0)
            a.call()
            assert ms.read_status(a.ws) == ms.STATUS_BAD_META and (a.out == 5.0).all(), (name, bad)
            setattr(a, name, old)
        total, a.total = a.total, a.total - 1  # a context sum above the call's bound
        a.call()
        assert ms.read_status(a.ws) == ms.STATUS_BAD_META
        a.total = total
        a.call()
        a.check()


def test_ragged_rows_short_of_pages(env):
    torch, ms, _ = env
    for window in (50, None):
        a = Span(env, [(100, 1), (64, 3)], 4, 2, 64, window, ragged=True)
        off = a.off.clone()
        a.off[1] -= 1
        a.call()
        assert ms.read_status(a.ws) == ms.STATUS_BAD_META and (a.out == 5.0).all()
        a.off.copy_(off)
        a.call()
        a.check()


def test_repeat_streams_and_replays_give_the_same_bits(env):
    """Two calls at once on two streams with a workspace each; the same captured, and replayed as lengths change."""
    torch, ms, _ = env
    a = Span(env, [(3000, 1), (500, 200), (8000, 1), (9000, 20)], 8, 2, 128, 2500, 1.0, seed=1)
    b = Span(env, [(9001, 20), (77, 1), (64, 300), (0, 4)], 4, 4, 64, None, seed=2)
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
    for x, w in zip((a, b), want):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            x.call(stream=streams[0])
        for _ in range(3):
            x.out.fill_(9.0)
            g.replay()
            assert torch.equal(x.out[:x.T], w[:x.T])
        # shorter rows in the same graph
        x.rows = [(max(c - 37, 0), d) for c, d in x.rows]
        x.ends = [c if x.cross else c + d for c, d in x.rows]
        x.first = [0 if x.cross else max(0, c + 1 - x.window) for c, _ in x.rows]
        if not x.cross:  # the pages that come back into the windows
            for s in range(len(x.rows)):
                x.pages[s][:] = x.pages[s][-1]
                x.bt[s, :len(x.pages[s])] = int(x.pages[s][-1])
            x.k.nan_to_num_(0, 0, 0)
            x.v.nan_to_num_(0, 0, 0)
        x.lens.copy_(_i32(torch, x.ends))
        x.start.copy_(_i32(torch, [c for c, _ in x.rows]))
        g.replay()
        x.check(out=torch.cat([x.out[:x.T], torch.full_like(x.out[x.T:], 5.0)]))


def test_long_rows(env):
    """A decode of 150000 keys (many splits, the sink in the first one only) and two tokens over as many, in parts."""
    for window, sinks in ((ALL, 2.0), (100001, None), (None, None)):
        a = Span(env, [(150000, 1), (149990, 2), (70000, 1)], 8, 2, 64, window, sinks, seed=11)
        a.call()
        a.check()


def test_page_ids_past_32_bit_offsets(env):
    """Pages whose elements lie past 2^31 from the pool's start."""
    torch, ms, _ = env
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    for window in (3000, None):
        a = Span(env, [(4000, 1), (500, 70)], 8, 8, 128, window, seed=2, poison=False)
        pages = 140000
        k, v = (torch.zeros(pages, 8, 16, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        n = a.k.shape[0]
        k[pages - n:], v[pages - n:] = a.k, a.v
        a.k, a.v = k, v
        a.pages = [p + pages - n for p in a.pages]
        a.bt[(a.bt >= 0) & (a.bt < n)] += pages - n
        a.call()
        a.check()
        del k, v


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("where", ["v above k", "v below k", "one pool for both", "side by side"])
def test_pools_in_any_place(env, H_q, H_kv, D, where):
    """A page of K and of V comes as one box where the pools' distance is one that a tensor map can have, whichever pool
    lies lower; one tensor as both pools comes as two.  Hidden cells of both hold infinities and NaN."""
    torch = env[0]
    for window in (70, None):
        a = Span(env, [(333, 130), (40, 1), (1000, 3), (17, 17), (2500, 1)], H_q, H_kv, D, window, 1.0 if window else None, seed=6)
        n = a.k.numel()
        if where == "one pool for both":
            a.v = a.k
        else:
            gap = {"side by side": 0, "v above k": 8 * 1234567, "v below k": 8 * 7}[where]
            both = torch.empty(2 * n + gap, dtype=torch.bfloat16, device="cuda")
            low, high = both[:n].view(a.k.shape), both[n + gap:].view(a.k.shape)
            k, v = (high, low) if where == "v below k" else (low, high)
            k.copy_(a.k)
            v.copy_(a.v)
            a.k, a.v = k, v
        a.call()
        a.check()


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (4, 4, 64), (8, 1, 64)])
@pytest.mark.parametrize("where,form", [("k first", 1), ("v first", 2), ("one pool", 0)])
def test_which_boxes_the_pages_came_in(env, H_q, H_kv, D, where, form):
    """The header says how a page of K and of V came: as one box with the lower pool's half first, or as two."""
    torch = env[0]
    for window in (70, None):
        a = Span(env, [(333, 130), (40, 1), (1000, 3), (17, 17)], H_q, H_kv, D, window, 1.0 if window else None, seed=12)
        n = a.k.numel()
        both = torch.empty(2 * n + 16, dtype=torch.bfloat16, device="cuda")
        if where == "one pool":
            a.v = a.k
        else:
            k, v = (both[n + 16:], both[:n]) if where == "v first" else (both[:n], both[n + 16:])
            a.k, a.v = k.view(a.k.shape).copy_(a.k), v.view(a.v.shape).copy_(a.v)
        a.call()
        a.check()
        assert a.word(KV_FORM) == form


@pytest.mark.parametrize("H_q,H_kv,D", [(8, 2, 128), (4, 4, 64)])
@pytest.mark.parametrize("rows", [[(500, 300), (20, 40)], [(9000, 20)]])
def test_stalled_producers_time_out_and_the_workspace_recovers(env, H_q, H_kv, D, rows):
    torch, ms, _ = env
    a = Span(env, rows, H_q, H_kv, D, ALL, seed=9)
    ms.test_attention_stall_window(a.q, a.k, a.v, a.cu, a.start, a.lens, a.bt, a.total, a.out, a.ws, ALL, 1000000)
    assert ms.read_status(a.ws) == ms.STATUS_TIMEOUT and (a.out == 5.0).all()
    a.call()
    a.check()


@pytest.mark.parametrize("seed", range(24))
def test_random_steps(env, seed):
    """Random rows, shapes, windows, sinks, tables and bounds on the contexts' sum, with and without the room for parts."""
    torch, ms, _ = env
    rng = np.random.default_rng(1000 + seed)
    G, H_kv, D = int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 2, 3, 5])), int(rng.choice([64, 128]))
    n = int(rng.choice([1, 2, 7, 40]))
    most = int(rng.choice([20, 300, 7000]))
    rows = [(int(rng.integers(0, most)), int(rng.choice([0, 1, 1, 1, 2, 5, 17, 130, 400])) if i < 6 else int(rng.choice([0, 1, 1, 1])))
            for i in range(n)]
    window = None if rng.random() < 0.3 else int(rng.choice([1, 2, 15, 16, 33, 64, 127, 500, 2000, ALL]))
    a = Span(env, rows, G * H_kv, H_kv, D, window, 2.0 if window and rng.random() < 0.5 else None, seed=seed, ragged=bool(rng.random() < 0.5),
             slack=int(rng.integers(0, 4)))
    scale = None if rng.random() < 0.7 else float(rng.uniform(0.02, 0.3))
    for q4 in (True, False):
        total = a.total + int(rng.integers(0, 500))
        ws = torch.zeros(ms.attention_workspace_size(n, a.q.shape[0], total, G * H_kv, H_kv, D, q4=q4), dtype=torch.uint8, device="cuda")
        a.out.fill_(5.0)
        a.total, keep = total, a.total
        a.call(scale, ws=ws)
        a.total = keep
        assert ms.read_status(ws) == 0
        a.check(scale)


# ---------------------------------------------------------------------------- together

@pytest.mark.parametrize("H_q,H_kv,D,R,interleaved,window", [(8, 2, 128, 64, True, 40), (4, 4, 64, 64, False, 17), (8, 1, 64, 16, True, None)])
def test_decoder_layer_captured(env, H_q, H_kv, D, R, interleaved, window):
    """Requests that prefill, then decode, through one captured step of two attentions: rows of a fused projection are
    appended with the rotation and attended to over a window with sinks, then the encoder's states are, which other pages
    hold.  The step's lengths change on the GPU; caches and outputs against the oracle and the plain forms."""
    torch, ms, step = env
    S, cap, pages, sinks = 3, 48, 60, torch.tensor(np.linspace(-2, 3, H_q), dtype=torch.float32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    enc = [0, 37, 150]
    ek, ev = (torch.zeros(14, H_kv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    states = [randn(sum(enc), H_kv, D) for _ in range(2)]
    ids = np.random.default_rng(1).permutation(14)
    ebt = np.full((S, 10), -1)
    ebt[1, :3], ebt[2] = ids[:3], ids[3:13]
    slots = [int(ebt[s, j // 16]) * 16 + j % 16 for s in range(S) for j in range(enc[s])]
    step.append_states(*states, _i32(torch, slots), ek, ev)
    kc, vc = (torch.zeros(pages, H_kv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    tables = step.StepTables(_i32(torch, np.random.default_rng(2).permutation(pages).reshape(S, 20)), pages, cap)
    cos, sin = step.rotary_tables(320, R, "cuda", scaling={"kind": "linear", "factor": 2.0})
    qkv, cq = randn(cap, H_q + 2 * H_kv, D), randn(cap, H_q, D)
    q, k, v = qkv.split([H_q, H_kv, H_kv], dim=1)
    q_rot, out, cout = (torch.empty(cap, H_q, D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    ws = torch.zeros(ms.attention_workspace_size(S, cap, 16 * pages, H_q, H_kv, D), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cached, new, key_lens, ebt_d = _i32(torch, [0, 0, 0]), _i32(torch, [0, 0, 0]), _i32(torch, enc), _i32(torch, ebt)

    def one(stream):
        batch = tables.build(cached, new, stream=stream)
        step.run_step(q, k, v, batch, cos, sin, kc, vc, out, ws, q_rot=q_rot, dev_status=status, interleaved=interleaved,
                      window=window, sinks=sinks, stream=stream)
        step.cross_attend(cq, ek, ev, batch, key_lens, ebt_d, sum(enc), cout, ws, stream=stream)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        one(s)
    c = [0, 0, 0]
    table = tables.page_tables.cpu().numpy()
    for d in ([20, 0, 3], [1, 33, 7], [1, 1, 46], [1, 0, 1], [20, 20, 1]):
        qkv.copy_(randn(*qkv.shape))
        cached.copy_(_i32(torch, c))
        new.copy_(_i32(torch, d))
        graph.replay()
        torch.cuda.synchronize()
        assert ms.read_status(status) == 0 and ms.read_status(ws) == 0 and ms.read_status(tables.status) == 0
        T = sum(d)
        pos = np.concatenate([np.arange(a, a + n) for a, n in zip(c, d)]).astype(int)
        tc, ts = cos.cpu().numpy()[pos], sin.cpu().numpy()[pos]
        np.testing.assert_array_equal(workloads.bf16_bits(q_rot[:T]), rotary.rotate(workloads.bf16_bits(q[:T].contiguous()), tc, ts, interleaved))
        kr = rotary.rotate(workloads.bf16_bits(k[:T].contiguous()), tc, ts, interleaved)
        t = 0
        for r in range(S):
            for i in range(d[r]):
                page, at = table[r, (c[r] + i) // 16], (c[r] + i) % 16
                np.testing.assert_array_equal(workloads.bf16_bits(kc[page, :, at]), kr[t])
                assert torch.equal(vc[page, :, at], v[t])
                t += 1
        a = Span(env, list(zip(c, d)), H_q, H_kv, D, ALL if window is None else window, poison=False)
        a.pages, a.k, a.v, a.q, a.sinks, a.ws = [row.astype(np.int64) for row in table], kc, vc, q_rot, sinks, ws
        a.check(out=out[:T])
        b = Span(env, list(zip(enc, d)), H_q, H_kv, D, None, poison=False)
        b.pages, b.k, b.v, b.q, b.ws = [row.astype(np.int64) for row in ebt], ek, ev, cq, ws
        b.check(out=cout[:T])
        c = [a0 + n for a0, n in zip(c, d)]


def test_run_step_picks_the_plain_step(env):
    """Without any form run_step is ms_mixed_step, bit for bit; the eager forms equal the separate calls."""
    torch, ms, step = env
    wl = workloads.worked_example()
    states = [(r.cached_len, r.remaining) for r in wl.requests]
    meta = ms.build_batch_metadata(states, [r.block_table for r in wl.requests], wl.token_budget)
    batch = step.to_device(meta, "cuda")
    T = meta["num_tokens"]
    q, k, v = workloads.step_tensors(wl, T, 1, "cuda")
    ws = step.workspace_for(batch, wl.H_q, wl.H_kv, wl.D, "cuda", q4=True)
    tabs = step.rope_tables_device(wl.max_pos + 1, wl.D, "cuda")
    res = []
    for call in range(2):
        kc, vc = workloads.kv_pool(wl, 1, "cuda")
        out, q_rot = torch.zeros_like(q), torch.empty_like(q)
        if call == 0:
            step.run_step(q, k, v, batch, *tabs, kc, vc, out, ws, q_rot=q_rot)
        else:
            ms.kv_append_rotary(q, k, v, batch.positions, batch.slot_mapping, *tabs, kc, vc, q_rot=q_rot)
            step.attend(q_rot, kc, vc, batch, out, ws)
        res.append((q_rot, kc, vc, out))
    assert all(torch.equal(x, y) for x, y in zip(*res))
    kc, vc = workloads.kv_pool(wl, 1, "cuda")
    out, q_rot = torch.zeros_like(q), torch.empty_like(q)
    step.run_step(q, k, v, batch, *tabs, kc, vc, out, ws, q_rot=q_rot, window=20)
    assert torch.equal(q_rot, res[0][0]) and torch.equal(kc, res[0][1]) and not torch.equal(out, res[0][3])
    assert ms.read_status(ws) == 0


@pytest.mark.parametrize("R", [32, 0])
def test_step_turns_the_part_of_the_head_that_it_is_told(env, R):
    """With rotary_dim given, halves of a part of the head, or nothing, turn: the separate calls' bits, eager and by rounds."""
    torch, ms, step = env
    from chunked_prefill_mixed_decode_gb300.driver import RoundDriver
    H_q, H_kv, D, budget, pages = 4, 2, 64, 24, 12
    g = torch.Generator(device="cuda").manual_seed(R)
    tabs = step.rotary_tables(200, R, "cuda") if R else (None, None)
    pools = [torch.zeros(pages, H_kv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    eng = ms.Engine(pages, budget)
    drv = RoundDriver(eng, pools[0], pools[1], *tabs, H_q, H_kv, D, rotary_dim=R)
    eng.add_request(37, 3)
    eng.add_request(5, 4)
    for _ in range(4):
        q, k, v = (torch.randn(budget, H, D, generator=g, device="cuda").to(torch.bfloat16) for H in (H_q, H_kv, H_kv))
        m = drv.step(q, k, v)["meta"]
        T = m["num_tokens"]
        assert T > 0
        batch = step.to_device(m, "cuda")
        ws = step.workspace_for(batch, H_q, H_kv, D, "cuda")
        q_rot, out = torch.empty(T, H_q, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, H_q, D, dtype=torch.bfloat16, device="cuda")
        ms.kv_append_rotary(q[:T], k[:T], v[:T], batch.positions, batch.slot_mapping, *tabs, pools[2], pools[3], q_rot=q_rot)
        step.attend(q_rot, pools[2], pools[3], batch, out, ws)
        assert torch.equal(drv.q_rot[:T], q_rot) and torch.equal(drv.out[:T], out)
        assert torch.equal(pools[0], pools[2]) and torch.equal(pools[1], pools[3])
        assert torch.equal(q_rot, q[:T]) == (R == 0)


@pytest.mark.parametrize("window,sinks", [(24, True), (None, True), (9, False)])
def test_engine_rounds_with_a_window(env, window, sinks):
    """The round driver over pools with pages reused: every round's windowed attention against the plain form."""
    torch, ms, step = env
    from chunked_prefill_mixed_decode_gb300.driver import RoundDriver
    H_q, H_kv, D, budget, pages = 8, 2, 64, 24, 24
    eng = ms.Engine(pages, budget)
    rng = np.random.default_rng(5)
    kc, vc = (torch.zeros(pages, H_kv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sk = torch.randn(H_q, device="cuda") if sinks else None
    cos, sin = step.rotary_tables(400, 32, "cuda")
    drv = RoundDriver(eng, kc, vc, cos, sin, H_q, H_kv, D, interleaved=True, window=window, sinks=sk)
    served = 0
    for _ in range(30):
        try:
            eng.add_request(int(rng.integers(1, 70)), int(rng.integers(1, 12)))
        except ms.MixedStepError as e:
            assert e.code == ms.MS_ERR_NO_PAGES
        q, k, v = (torch.randn(budget, H, D, device="cuda").to(torch.bfloat16) for H in (H_q, H_kv, H_kv))
        rec = drv.step(q, k, v)
        m = rec["meta"]
        if m["num_tokens"] == 0:
            continue
        served += 1
        rows = [(int(c), int(b - a)) for c, a, b in zip(m["q_start_pos"], m["cu_seqlens_q"], m["cu_seqlens_q"][1:])]
        a = Span(env, rows, H_q, H_kv, D, ALL if window is None else window, poison=False)
        a.pages, a.k, a.v, a.q, a.sinks, a.ws = [r.astype(np.int64) for r in m["block_tables"]], kc, vc, drv.q_rot, sk, drv.workspace
        a.check(out=drv.out[:m["num_tokens"]])
    assert served > 20
