"""The rotary table and the append in their other forms, on the GPU, against the oracle.

A table entry is off by at most 0.8 of a step of fp32 (a step of v is at most 2^-23 |v|; the definition of the kernel's
arithmetic gives 0.5 for the last rounding and 0.28 for the cubic term's) and by the error of its angle: 2^-65 turns a
position, and the first Taylor terms left out, 3e-9.  The append is compared bit for bit.
"""
import numpy as np
import pytest

import oracle
import workloads
from oracle import rotary

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


# ---------------------------------------------------------------------------- table

SCALINGS = [None, {"kind": "linear", "factor": 4.0}, {"kind": "base", "factor": 8.0},
            {"kind": "bands", "factor": 8.0, "original_len": 8192, "low": 1.0, "high": 4.0},
            {"kind": "ramp", "factor": 4.0, "original_len": 32768, "low": 1.0, "high": 32.0}]


def _check_table(env, freq, amp, first, n, rows=None, row_len=None):
    torch, ms, _ = env
    pairs = len(freq)
    cos, sin = (torch.full((n + 2, pairs), 7.0, device="cuda") for _ in range(2))  # and two rows that are not its own
    ms.rotary_table_device(freq, cos[:n], sin[:n], amplitude=amp, first_pos=first)
    assert (cos[n:] == 7.0).all() and (sin[n:] == 7.0).all()
    rows = range(n) if rows is None else rows
    for r in rows:
        want = np.array([rotary.table_entry(first + r, f, amp) for f in freq])
        for got, w in ((cos[r], want[:, 0]), (sin[r], want[:, 1])):
            bound = 0.8 * 2.0 ** -23 * np.abs(w) + abs(amp) * (2 * np.pi * (first + r + 1) * 2.0 ** -65 + 3e-9)
            assert (np.abs(got.cpu().numpy().astype(np.float64) - w) <= bound).all(), (first + r)


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("R,base,first,n", [(128, 10000.0, 0, 130), (16, 10000.0, 0, 1), (48, 500000.0, 4093, 70), (64, 1e6, 131071, 33),
                                            (96, 10000.0, 10 ** 6, 40), (128, 10000.0, 2 ** 31 - 20, 20), (24, 100.0, 77, 500)])
def test_table(env, R, base, first, n, scaling):
    freq, amp = env[1].rotary_frequencies(R, base, scaling)
    _check_table(env, freq, amp, first, n, rows=sorted({0, 1, 2, n // 3, n // 2, n - 2, n - 1} & set(range(n))))


@pytest.mark.parametrize("R,base,factor,amp", [(128, 1e6, 32.0, 1.0), (128, 5e5, 8.0, 1.0), (128, 1e4, 1.0, 1.1386), (64, 1e4, 4.0, -2.5),
                                               (128, 1e6, 1.0, 1.41)])
@pytest.mark.parametrize("first,n", [(0, 12), (4095, 4), (2 ** 20 - 2, 4), (2 ** 31 - 4, 4)])
def test_table_entry_by_entry(env, R, base, factor, amp, first, n):
    """Every entry, the smallest sines among them, against the arithmetic's own error and nothing beside it.

    Of the value's size, in units of 2^-23: 0.5 for the last rounding; 3.5 roundings of 2^-24 in the cubic term, at most
    0.115 of a sine up to pi / 4: 0.2; the first term left out, x^11 / 11! or x^12 / 12!, 0.02; 0.005 for the fifth
    power's: 0.73 in all, 0.8 here.  Of the angle: (p + 1) 2^-65 turns from the frequency's last bit and the product; what the
    series takes of the rest of the turn, 2 pi 2^-47 for the bits left out below it, and roundings of its small part of 2 pi
    2^-48 and 2^-49 at most: 2 pi 2^-46 in all.  (A step-by-step emulation in fp32 comes to 0.73 of this bound.)"""
    torch, ms, _ = env
    freq, _ = ms.rotary_frequencies(R, base, {"kind": "linear", "factor": factor})
    cos, sin = (torch.empty(n, R // 2, device="cuda") for _ in range(2))
    ms.rotary_table_device(freq, cos, sin, amplitude=amp, first_pos=first)
    for r in range(n):
        want = np.array([rotary.table_entry(first + r, f, amp) for f in freq])
        for got, w in ((cos[r], want[:, 0]), (sin[r], want[:, 1])):
            bound = 0.8 * 2.0 ** -23 * np.abs(w) + abs(amp) * 2 * np.pi * ((first + r + 1) * 2.0 ** -65 + 2.0 ** -46)
            assert (np.abs(got.cpu().numpy().astype(np.float64) - w) <= bound).all(), first + r


def test_table_of_special_angles(env):
    """Zero, negative and large frequencies, exact quarters' neighbourhood, a negative and a zero amplitude."""
    f = np.array([0.0, -0.7, 1024.0, -1024.0, np.pi / 2, np.pi / 4, -np.pi, 2 * np.pi, 1e-300, 1e-12, 5e-324, 0.5])
    _check_table(env, f, 1.0, 0, 40)
    _check_table(env, f, -2.5, 5, 8)
    _check_table(env, f, 0.0, 5, 3)


def test_long_table_against_another_reduction(env):
    """131072 rows: every entry against fp64 sines of fp64 products (their angles' rounding: 2^17 * 2^-53)."""
    torch, ms, step = env
    for scaling in (None, SCALINGS[4]):
        cos, sin = step.rotary_tables(131072, 128, "cuda", scaling=scaling)
        freq, amp = ms.rotary_frequencies(128, 10000.0, scaling)
        ang = torch.arange(131072, dtype=torch.float64, device="cuda")[:, None] * torch.tensor(freq, device="cuda")
        for got, w in ((cos, ang.cos() * amp), (sin, ang.sin() * amp)):
            assert ((got.double() - w).abs() <= 0.8 * 2.0 ** -23 * w.abs() + amp * (2.0 ** -36 + 3e-9)).all()


def test_table_replayed_and_refused(env):
    torch, ms, step = env
    f, _ = ms.rotary_frequencies(64)
    a, b = (torch.empty(100, 32, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ms.rotary_table_device(f, a, b, first_pos=50, stream=s)
    f[:] = 0  # read before the call returned
    a.zero_()
    g.replay()
    want = step.rotary_tables(100, 64, "cuda", first_pos=50)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])
    with pytest.raises(ms.MixedStepError):
        ms.rotary_table_device(np.zeros(6), a[:, :6].contiguous(), b[:, :6].contiguous())
    with pytest.raises(ms.MixedStepError):
        ms.rotary_table_device(np.zeros(32), a.view(-1)[1:3169].view(99, 32), b[:99])
    ms.rotary_table_device(np.zeros(32), a[:0], b[:0])


# ---------------------------------------------------------------------------- append

def _inputs(torch, T, H_q, H_kv, D, seed, fused):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        x = torch.randn(T, H_q + 2 * H_kv + 1, D, generator=g, device="cuda").to(torch.bfloat16)
        return x[:, :H_q], x[:, H_q:H_q + H_kv], x[:, H_q + H_kv:H_q + 2 * H_kv]
    return [torch.randn(T, H, D, generator=g, device="cuda").to(torch.bfloat16) for H in (H_q, H_kv, H_kv)]


def _run(env, q, k, v, positions, slots, tabs, interleaved, pages, q_rot=None):
    """The call on pools of sevens; (q_rot, k pool, v pool) as bits, and the status."""
    torch, ms, _ = env
    H_kv, D = k.shape[1:]
    kc, vc = (torch.full((pages, H_kv, 16, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if q is not None and q_rot is None:
        q_rot = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    cos, sin = tabs if tabs is not None else (None, None)
    ms.kv_append_rotary(q, k, v, None if positions is None else _i32(torch, positions), _i32(torch, slots), cos, sin, kc, vc,
                        q_rot=q_rot, interleaved=interleaved, dev_status=status)
    return None if q is None else workloads.bf16_bits(q_rot), workloads.bf16_bits(kc), workloads.bf16_bits(vc), ms.read_status(status)


def _want(torch, q, k, v, positions, slots, tabs, interleaved, pages, ok):
    H_kv, D = k.shape[1:]
    bits = [None if x is None else workloads.bf16_bits(x.contiguous()) for x in (q, k, v)]
    if tabs is not None:
        cos, sin = (x.cpu().numpy()[np.clip(positions, 0, len(x) - 1)] for x in tabs)
        bits[:2] = [None if x is None else rotary.rotate(x, cos, sin, interleaved) for x in bits[:2]]
    kp, vp = (np.full((pages, H_kv, 16, D), 0x40E0, dtype=np.uint16) for _ in range(2))
    for t, s in enumerate(slots):
        if ok[t]:
            kp[s // 16, :, s % 16], vp[s // 16, :, s % 16] = bits[1][t], bits[2][t]
    return bits[0], kp, vp


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H_q,H_kv,D,R,T,fused", [(4, 2, 64, 64, 1, False), (4, 2, 64, 32, 37, True), (8, 1, 64, 16, 5, True),
                                                  (32, 8, 128, 128, 33, True), (32, 32, 128, 64, 9, False), (5, 3, 128, 48, 50, True),
                                                  (1, 1, 128, 112, 300, True), (7, 2, 64, 48, 19, False), (40, 40, 128, 16, 3, True),
                                                  (3, 5, 64, 64, 1000, True)])
def test_append(env, H_q, H_kv, D, R, T, fused, interleaved):
    """Bit for bit, over random slots; cells that no token names and gaps between fused rows keep what they held."""
    torch, ms, step = env
    rng = np.random.default_rng(T + R)
    q, k, v = _inputs(torch, T, H_q, H_kv, D, T + D, fused)
    pages = 2 * (-(-T // 16)) + 1
    slots, positions = rng.permutation(16 * pages)[:T], rng.integers(0, 5000, T)
    tabs = step.rotary_tables(5000, R, "cuda")
    got = _run(env, q, k, v, positions, slots, tabs, interleaved, pages)
    assert got[3] == 0
    for g, w in zip(got, _want(torch, q, k, v, positions, slots, tabs, interleaved, pages, [True] * T)):
        np.testing.assert_array_equal(g, w)


@pytest.mark.parametrize("D,T,H_q", [(64, 1, 0), (64, 100, 4), (128, 333, 0), (128, 17, 8)])
def test_append_without_rotation(env, D, T, H_q):
    """An encoder's states as they are, NaN and infinities among them; with q, which is copied."""
    torch = env[0]
    q, k, v = _inputs(torch, T, max(H_q, 1), 3, D, T, T % 2 == 0)
    k[T // 2, 1, 3], v[T - 1, 2, 5], v[0, 0, 0] = float("nan"), float("inf"), -0.0
    q = q if H_q else None
    pages = -(-T // 16) + 1
    slots = np.random.default_rng(T).permutation(16 * pages)[:T]
    got = _run(env, q, k, v, None, slots, None, False, pages)
    assert got[3] == 0
    for g, w in zip(got, _want(torch, q, k, v, None, slots, None, False, pages, [True] * T)):
        if w is not None:
            np.testing.assert_array_equal(g, w)


@pytest.mark.parametrize("D", [64, 128])
def test_whole_head_in_halves_is_the_plain_append(env, D):
    """Bit for bit, host-made tables, and in place."""
    torch, ms, step = env
    T, H_q, H_kv, pages = 200, 8, 2, 20
    rng = np.random.default_rng(3)
    q, k, v = _inputs(torch, T, H_q, H_kv, D, 5, False)
    slots, positions = _i32(torch, rng.permutation(16 * pages)[:T]), _i32(torch, rng.integers(0, 3000, T))
    cos, sin = step.rope_tables_device(3000, D, "cuda")
    res = []
    for call in (ms.kv_append_rope, ms.kv_append_rotary):
        kc, vc = (torch.zeros(pages, H_kv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        qq = q.clone()
        call(qq, k, v, positions, slots, cos, sin, kc, vc)
        res.append((qq, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_append_bad_slots_and_positions(env):
    torch = env[0]
    D, H_q, H_kv, pages = 64, 4, 2, 3
    q, k, v = _inputs(torch, 6, H_q, H_kv, D, 1, True)
    tabs = env[2].rotary_tables(10, 32, "cuda")
    for slots, positions, flag in (([0, -1, 47, 5, -1, 9], [1] * 6, 0), ([0, 48, 47, 5, 6, 9], [1] * 6, 1),
                                   ([0, -2, 47, 5, 6, 9], [1] * 6, 1), ([0, 1, 2, 3, 4, 5], [0, 9, 10, 3, -1, 2], 2),
                                   ([0, 1, 99, 3, 4, 5], [0, 9, 10, 3, 1, 2], 3)):
        for interleaved in (False, True):
            got = _run(env, q, k, v, positions, slots, tabs, interleaved, pages)
            assert got[3] == flag
            in_table = [0 <= p < 10 for p in positions]
            ok = [0 <= s < 16 * pages and i for s, i in zip(slots, in_table)]
            want = _want(torch, q, k, v, positions, slots, tabs, interleaved, pages, ok)
            for t in range(6):  # a token outside the table writes nothing at all
                np.testing.assert_array_equal(got[0][t], want[0][t] if in_table[t] else np.full_like(got[0][t], 0x40E0))
            np.testing.assert_array_equal(got[1], want[1])
            np.testing.assert_array_equal(got[2], want[2])


def test_append_of_no_token_and_without_status(env):
    torch, ms, step = env
    q, k, v = _inputs(torch, 4, 2, 1, 64, 2, False)
    kc, vc = (torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cos, sin = step.rotary_tables(8, 64, "cuda")
    i = _i32(torch, [0, 1, 2, 99])
    ms.kv_append_rotary(q[:0], k[:0], v[:0], i, i, cos, sin, kc, vc)
    assert not kc.any()
    ms.kv_append_rotary(q, k, v, i, i, cos, sin, kc, vc)  # the last token's slot and position are bad, and not reported
    torch.cuda.synchronize()
    assert vc[0, 0, :3].any(-1).all() and not vc[0, 0, 3:].any()


def test_append_past_32_bit_offsets(env):
    """Rows of q, and cells of the pools, more than 2^31 elements from the first."""
    torch, ms, step = env
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    D, H_kv, pages = 128, 8, 135000  # 2.2e9 elements a pool
    base = torch.zeros(3, 1 << 30, dtype=torch.bfloat16, device="cuda")
    q = base[:, :2 * D].unflatten(1, (2, D))
    q.normal_()
    k, v = (torch.randn(3, H_kv, D, device="cuda").to(torch.bfloat16) for _ in range(2))
    kc, vc = (torch.zeros(pages, H_kv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots, positions = [16 * pages - 1, 16 * 131073 + 5, 0], [7, 0, 3]
    tabs = step.rotary_tables(8, 64, "cuda")
    q_rot = torch.empty(3, 2, D, dtype=torch.bfloat16, device="cuda")
    ms.kv_append_rotary(q, k, v, _i32(torch, positions), _i32(torch, slots), *tabs, kc, vc, q_rot=q_rot, interleaved=True)
    cos, sin = (x.cpu().numpy()[positions] for x in tabs)
    np.testing.assert_array_equal(workloads.bf16_bits(q_rot), rotary.rotate(workloads.bf16_bits(q.contiguous()), cos, sin, True))
    kr = rotary.rotate(workloads.bf16_bits(k), cos, sin, True)
    for t, s in enumerate(slots):
        np.testing.assert_array_equal(workloads.bf16_bits(kc[s // 16, :, s % 16]), kr[t])
        assert torch.equal(vc[s // 16, :, s % 16], v[t])
    assert int((vc != 0).any(-1).sum()) == 3 * H_kv


def test_append_on_another_stream_and_replayed(env):
    torch, ms, step = env
    T, H_q, H_kv, D, pages = 70, 8, 4, 128, 9
    q, k, v = _inputs(torch, T, H_q, H_kv, D, 9, True)
    tabs = step.rotary_tables(300, 96, "cuda")
    rng = np.random.default_rng(0)
    slots, pos = _i32(torch, rng.permutation(16 * pages)[:T]), _i32(torch, rng.integers(0, 300, T))
    kc, vc = (torch.zeros(pages, H_kv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q_rot = torch.empty(T, H_q, D, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ms.kv_append_rotary(q, k, v, pos, slots, *tabs, kc, vc, q_rot=q_rot, stream=s)
    for shift in (0, 13):  # other positions and values, the same graph
        pos += shift
        pos %= 300
        q += shift
        g.replay()
        torch.cuda.synchronize()
        cos, sin = (x.cpu().numpy()[pos.cpu().numpy()] for x in tabs)
        np.testing.assert_array_equal(workloads.bf16_bits(q_rot), rotary.rotate(workloads.bf16_bits(q.contiguous()), cos, sin, False))
