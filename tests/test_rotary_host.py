"""Scaled rotary frequencies, and what the rotary, windowed and cross-attention calls refuse (CPU)."""
import ctypes
import math

import numpy as np
import pytest

import oracle
from oracle import rotary


@pytest.fixture(scope="module")
def ms():
    from chunked_prefill_mixed_decode_gb300 import build
    build.build()
    import chunked_prefill_mixed_decode_gb300 as ms
    return ms


SCALINGS = [None, {"kind": "plain"}, {"kind": "linear", "factor": 4.0}, {"kind": "base", "factor": 8.0},
            {"kind": "bands", "factor": 8.0, "original_len": 8192, "low": 1.0, "high": 4.0},
            {"kind": "ramp", "factor": 4.0, "original_len": 32768, "low": 1.0, "high": 32.0},
            {"kind": "ramp", "factor": 0.5, "original_len": 4096, "low": 1.0, "high": 32.0},
            {"kind": "ramp", "factor": 40.0, "original_len": 4096, "low": 1.0, "high": 32.0, "amplitude": 1.25}]


@pytest.mark.parametrize("scaling", SCALINGS)
@pytest.mark.parametrize("R,base", [(128, 10000.0), (64, 500000.0), (48, 10000.0), (16, 1e6)])
def test_frequencies(ms, R, base, scaling):
    """Doubles from a few roundings each: 16 of them at most (powers and logarithms are within two)."""
    got, amp = ms.rotary_frequencies(R, base, scaling)
    want, wamp = rotary.frequencies(R, base, scaling)
    np.testing.assert_allclose(got, want, rtol=16 * 2.0 ** -52)
    assert abs(amp - wamp) <= 2.0 ** -50


def test_frequencies_by_hand(ms):
    """R = 4, base 100: 1 and 0.1.  Doubling the base's exponent range, dividing, and both ends of bands and ramp."""
    np.testing.assert_allclose(ms.rotary_frequencies(4, 100.0)[0], [1, 0.1], rtol=1e-15)
    np.testing.assert_allclose(ms.rotary_frequencies(4, 100.0, {"kind": "base", "factor": 10.0})[0], [1, 0.01], rtol=1e-15)
    # bands: 628.3 positions are 100 turns of pair 0 and 10 of pair 1; between 1 and 19 turns pair 1 keeps half
    sc = {"kind": "bands", "factor": 5.0, "original_len": 0, "low": 1.0, "high": 19.0}
    sc["original_len"] = 628
    keep = (628 * 0.1 / (2 * math.pi) - 1) / 18
    np.testing.assert_allclose(ms.rotary_frequencies(4, 100.0, sc)[0], [1, 0.1 * (keep + (1 - keep) / 5)], rtol=1e-14)
    # ramp: every pair turns more than 20 times over 10^6 positions, none less than once over 6
    assert ms.rotary_frequencies(4, 100.0, {**sc, "kind": "ramp", "original_len": 10 ** 6, "high": 20.0})[0][1] == pytest.approx(0.1)
    assert ms.rotary_frequencies(4, 100.0, {**sc, "kind": "ramp", "original_len": 1})[0] == pytest.approx([1, 0.02])
    # ... and none of 64 pairs even a sixth of a turn: all but the first are stretched
    f = ms.rotary_frequencies(128, 10000.0)[0]
    np.testing.assert_allclose(ms.rotary_frequencies(128, 10000.0, {**sc, "kind": "ramp", "original_len": 1})[0][1:], f[1:] / 5, rtol=1e-14)


def test_plain_frequencies_are_those_of_the_host_table(ms):
    cos, sin = ms.rope_table(300, 64)
    f, _ = ms.rotary_frequencies(64)
    for p, i in ((0, 0), (1, 0), (299, 31), (200, 5)):
        assert cos[p, i] == np.float32(math.cos(p * f[i])) and sin[p, i] == np.float32(math.sin(p * f[i]))


def test_exact_reduction_of_the_oracle():
    """Against the C library, whose reduction of an exactly representable angle is exact: powers of two as frequencies."""
    for p, e in ((1, 0), (7, 3), (2 ** 31 - 1, 0), (2 ** 31 - 1, 12), (123456789, 20)):
        c, s = rotary.table_entry(p, 2.0 ** -e)
        assert abs(c - math.cos(p * 2.0 ** -e)) < 1e-15 and abs(s - math.sin(p * 2.0 ** -e)) < 1e-15


def test_rotation_of_the_oracle():
    """Whole heads in halves are rope_rotate's; pairs are the halves' result with the elements in another order."""
    rng = np.random.default_rng(0)
    x = oracle.f32_to_bf16_bits(rng.standard_normal((5, 3, 64)))
    cos, sin = oracle.rope_tables([0, 1, 5, 100, 4095], 64)
    np.testing.assert_array_equal(rotary.rotate(x, cos, sin, False), oracle.rope_rotate(x, cos, sin))
    order = np.r_[np.arange(32) * 2, np.arange(32) * 2 + 1]
    np.testing.assert_array_equal(rotary.rotate(x, cos, sin, True)[..., order], oracle.rope_rotate(x[..., order], cos, sin))
    part = rotary.rotate(x, cos[:, :16], sin[:, :16], False)
    np.testing.assert_array_equal(part[..., 32:], x[..., 32:])
    np.testing.assert_array_equal(part[..., :32], rotary.rotate(x[..., :32].copy(), cos[:, :16], sin[:, :16], False))


def test_frequency_refusals(ms):
    one = np.zeros(64)
    amp = ctypes.c_double()
    call = ms.lib().ms_rotary_frequencies
    ok = ms.RotaryScaling(ms.ROTARY_RAMP, 4096, 4.0, 1.0, 32.0, 0.0)
    assert call(128, 10000.0, ctypes.byref(ok), one.ctypes.data, ctypes.addressof(amp)) == ms.MS_OK
    for R, base, sc in ((3, 1e4, None), (0, 1e4, None), (130, 1e4, None), (64, 0.0, None), (64, float("nan"), None),
                        (64, float("inf"), None), (64, 1e4, (5, 0, 1.0, 0, 0, 0)), (64, 1e4, (-1, 0, 1.0, 0, 0, 0)),
                        (64, 1e4, (1, 0, 0.0, 0, 0, 0)), (64, 1e4, (1, 0, float("nan"), 0, 0, 0)), (2, 1e4, (2, 0, 2.0, 0, 0, 0)),
                        (64, 1e4, (3, 0, 2.0, 1, 4, 0)), (64, 1e4, (3, 100, 2.0, 0, 4, 0)), (64, 1e4, (3, 100, 2.0, 4, 4, 0)),
                        (64, 1.0, (4, 100, 2.0, 1, 4, 0)), (64, 1e4, (4, 100, 2.0, 1, 4, -1.0))):
        s = None if sc is None else ctypes.byref(ms.RotaryScaling(*sc))
        assert call(R, base, s, one.ctypes.data, ctypes.addressof(amp)) == ms.MS_ERR_ARG, (R, base, sc)
    assert call(64, 1e4, None, None, ctypes.addressof(amp)) == ms.MS_ERR_ARG
    assert call(64, 1e4, None, one.ctypes.data, None) == ms.MS_ERR_ARG
    for bad in ({"kind": "yes"}, {"factor": 2.0}, {"kind": "linear"}, {"kind": "plain", "factor": 2.0},
                {"kind": "bands", "factor": 2.0, "original_len": 100, "low": 1.0},
                {"kind": "linear", "factor": 2.0, "amplitude": 1.0}):
        with pytest.raises(ValueError):
            ms.rotary_frequencies(64, 1e4, bad)
    with pytest.raises(ms.MixedStepError):
        ms.rotary_frequencies(64, 1e4, {"kind": "linear", "factor": -2.0})


def test_frequencies_beyond_what_doubles_hold_are_refused(ms):
    """A base or factor whose frequencies overflow gives an error and not infinities, NaN or zeros; nothing is written."""
    f, amp = np.full(64, 7.0), ctypes.c_double(7.0)
    call = ms.lib().ms_rotary_frequencies
    tiny = 1e-320
    for base, sc in ((1e300, (2, 0, 1e30, 0, 0, 0)), (1e-300, (2, 0, 1e-30, 0, 0, 0)), (1e4, (1, 0, tiny, 0, 0, 0)),
                     (1e4, (3, 8192, tiny, 1, 4, 0)), (1e4, (4, 8192, tiny, 1, 4, 0)), (5e-324, None)):
        s = None if sc is None else ctypes.byref(ms.RotaryScaling(*sc))
        assert call(64, base, s, f.ctypes.data, ctypes.addressof(amp)) == ms.MS_ERR_ARG, (base, sc)
        assert (f == 7.0).all() and amp.value == 7.0
    assert call(64, 1e300, ctypes.byref(ms.RotaryScaling(2, 0, 1e3, 0, 0, 0)), f.ctypes.data, ctypes.addressof(amp)) == ms.MS_OK
    assert np.isfinite(f).all() and (f[:32] > 0).all()


P = 4096  # an aligned address that no refused call may touch


def test_table_refusals(ms):
    f = np.full(64, 0.5)
    call = ms.lib().ms_rotary_table_device
    good = dict(freq=f.ctypes.data, pairs=64, amp=1.0, first=0, n=10, cos=P, sin=P)
    inf = np.full(64, np.inf)
    big = np.full(64, 1025.0)
    for change in ({"freq": None}, {"pairs": 0}, {"pairs": 6}, {"pairs": 68}, {"amp": float("nan")}, {"first": -1}, {"n": -1},
                   {"first": 2 ** 31 - 5}, {"cos": None}, {"sin": P + 4}, {"freq": inf.ctypes.data}, {"freq": big.ctypes.data},
                   {"amp": 1e31}, {"amp": 1e-13}, {"amp": float("inf")}):
        a = {**good, **change}
        assert call(a["freq"], a["pairs"], a["amp"], a["first"], a["n"], a["cos"], a["sin"], None) == ms.MS_ERR_ARG, change
    assert call(f.ctypes.data, 64, 1.0, 0, 0, None, None, None) == ms.MS_OK  # no rows


def test_append_refusals(ms):
    call = ms.lib().ms_kv_append_rotary
    names = ("q qs k ks v vs positions slots T cos sin max_pos R inter kc vc pages q_rot H_q H_kv D page status stream").split()
    good = dict(q=P, qs=512, k=P, ks=128, v=P, vs=128, positions=P, slots=P, T=3, cos=P, sin=P, max_pos=10, R=64, inter=0, kc=P,
                vc=P, pages=2, q_rot=2 * P, H_q=8, H_kv=2, D=64, page=16, status=None, stream=None)
    for change in ({"T": -1}, {"H_q": -1}, {"H_kv": 0}, {"D": 96}, {"page": 32}, {"pages": -1}, {"R": 8}, {"R": 80}, {"R": -16},
                   {"inter": 2}, {"max_pos": 0}, {"qs": 511}, {"qs": 504}, {"qs": 516}, {"ks": 120}, {"vs": 0}, {"vs": -128},
                   {"k": None}, {"v": P + 2}, {"kc": P + 8}, {"vc": None}, {"slots": None}, {"q": None}, {"q_rot": None},
                   {"q_rot": P + 8}, {"positions": None}, {"cos": None}, {"sin": P + 4}, {"qs": 640, "q_rot": P}):
        a = {**good, **change}
        assert call(*[a[n] for n in names]) == ms.MS_ERR_ARG, change
    for change in ({"T": 0}, {"T": 0, "k": None, "q": None}):
        a = {**good, **change}
        assert call(*[a[n] for n in names]) == ms.MS_OK, change


def test_attention_refusals(ms):
    window, cross = ms.lib().ms_mixed_step_attention_window, ms.lib().ms_mixed_step_cross_attention
    stall = ms.lib().ms_test_attention_stall_window
    wn = "q kc vc pages cu start lens bt off bt_len stride rows tokens total H_q H_kv D page scale window sinks out ws bytes stream".split()
    cn = [n for n in wn if n not in ("start", "window", "sinks")]
    sn = [n for n in wn if n not in ("off", "bt_len", "sinks", "stream")] + ["limit", "stream"]
    good = dict(q=P, kc=P, vc=P, pages=4, cu=P, start=P, lens=P, bt=P, off=None, bt_len=0, stride=4, rows=2, tokens=5, total=50,
                H_q=8, H_kv=2, D=64, page=16, scale=0.125, window=16, sinks=None, out=P, ws=P, bytes=1 << 30, stream=None,
                limit=1000000)
    both = [{"rows": -1}, {"tokens": -1}, {"total": -1}, {"H_q": 7}, {"H_q": 32}, {"H_q": 6, "H_kv": 2}, {"D": 32}, {"page": 8},
            {"scale": 0.0}, {"scale": float("nan")}, {"stride": -1}, {"pages": -1}, {"q": None}, {"kc": P + 8}, {"vc": None},
            {"cu": None}, {"lens": None}, {"bt": None}, {"stride": 0}, {"out": None}, {"ws": P + 128}, {"ws": None}, {"bytes": 1000},
            {"off": P, "bt_len": 0}, {"rows": 8193}, {"tokens": (1 << 21) + 1}]
    for change in both + [{"window": 0}, {"window": -5}, {"sinks": P + 2}, {"start": None}]:
        a = {**good, **change}
        assert window(*[a[n] for n in wn]) == ms.MS_ERR_ARG, change
    for change in both:
        a = {**good, **change}
        assert cross(*[a[n] for n in cn]) == ms.MS_ERR_ARG, change
    for change in ({"window": 0}, {"limit": 0}, {"limit": 1 << 40}, {"q": None}):
        a = {**good, **change}
        assert stall(*[a[n] for n in sn]) == ms.MS_ERR_ARG, change
    for empty in ({"rows": 0}, {"tokens": 0}):  # nothing to do, nothing enqueued
        a = {**good, **empty}
        assert window(*[a[n] for n in wn]) == ms.MS_OK and cross(*[a[n] for n in cn]) == ms.MS_OK


def test_binding_refusals(ms):
    """What the C side cannot see: types, shapes, layouts, devices."""
    torch = pytest.importorskip("torch")
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    T, H_q, H_kv, D = 4, 4, 2, 64
    k, v = torch.zeros(T, H_kv, D, dtype=bf), torch.zeros(T, H_kv, D, dtype=bf)
    q, pos = torch.zeros(T, H_q, D, dtype=bf), torch.zeros(T, dtype=i32)
    cos = torch.zeros(10, 16, dtype=f32)
    pool = torch.zeros(3, H_kv, 16, D, dtype=bf)
    good = dict(q=q, k=k, v=v, positions=pos, slot_mapping=pos, cos_tab=cos, sin_tab=cos.clone(), k_cache=pool, v_cache=pool.clone())
    wide = torch.zeros(T, H_kv, 2 * D, dtype=bf)
    for change in ({"k": None}, {"k": k[0]}, {"k": k.float()}, {"k": wide[..., ::2]}, {"k": wide[..., :D]}, {"v": v[:2]},
                   {"q": q[:2]}, {"q": q[..., :32]}, {"q_rot": q.float()}, {"q": None, "q_rot": q}, {"cos_tab": None},
                   {"cos_tab": cos.double()}, {"sin_tab": cos[:5]}, {"positions": pos[:2]}, {"positions": pos.long()},
                   {"slot_mapping": pos[:1]}, {"k_cache": pool[0]}, {"v_cache": pool[:2]}, {"k_cache": None},
                   {"q": torch.zeros(T, 2 * H_q, D, dtype=bf)[:, :H_q]},  # in place with gaps
                   {"dev_status": pos.float()}, {}):  # {}: not on a GPU
        with pytest.raises(ValueError):
            ms.kv_append_rotary(**{**good, **change})
    cu = torch.zeros(3, dtype=i32)
    a = dict(q_rot=q, k_cache=pool, v_cache=pool.clone(), cu_seqlens_q=cu, q_start_pos=cu, context_lens=cu, out=q.clone(),
             block_tables=torch.zeros(2, 3, dtype=i32), context_total=4, workspace=torch.zeros(1 << 16, dtype=torch.uint8), window=4)
    for change in ({"q_rot": q.float()}, {"q_rot": q[0]}, {"k_cache": pool.float()}, {"cu_seqlens_q": cu.long()}, {"q_start_pos": cu[:1]},
                   {"context_lens": None}, {"block_tables": cu[:1].view(1, 1).expand(2, 3)}, {"bt_offsets": cu[:2]},
                   {"sinks": torch.zeros(H_q - 1)}, {"sinks": torch.zeros(H_q, dtype=torch.float64)}, {"out": q[:2]}, {"workspace": None}, {}):
        with pytest.raises((ValueError, AttributeError)):
            ms.mixed_step_attention_window(**{**a, **change})
    c = dict(q=q, k_cache=pool, v_cache=pool.clone(), cu_seqlens_q=cu, key_lens=cu, block_tables=a["block_tables"], key_total=4,
             out=q.clone(), workspace=a["workspace"])
    for change in ({"key_lens": cu[:1]}, {"key_lens": cu.float()}, {"out": q.float()}, {}):
        with pytest.raises(ValueError):
            ms.mixed_step_cross_attention(**{**c, **change})
    for change in ({"freq": np.zeros(8)}, {"cos_tab": cos.view(-1)}, {"sin_tab": cos.double()}, {}):
        with pytest.raises(ValueError):
            ms.rotary_table_device(**{"freq": np.zeros(16), "cos_tab": cos, "sin_tab": cos.clone(), **change})


def test_round_driver_refuses_forms_without_their_kernels(ms):
    torch = pytest.importorskip("torch")
    from chunked_prefill_mixed_decode_gb300.driver import RoundDriver
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    q4 = torch.zeros(2, 2, 18 * 64, dtype=torch.uint8)
    for kw in ({"interleaved": True}, {"window": 8}, {"sinks": torch.zeros(4)}):
        with pytest.raises(ValueError):
            RoundDriver(ms.Engine(2, 8), q4, None, None, None, 4, 2, 64, **kw)
        with pytest.raises(ValueError):
            RoundDriver(ms.Engine(2, 8), pool, pool, None, None, 4, 2, 64, graph_buckets=[8], **kw)


def _host_step(ms, D=128, H_q=4, H_kv=2, T=3):
    """Arguments of step.run_step on the host: what is refused by shape alone is refused before a device is looked for."""
    torch = pytest.importorskip("torch")
    from chunked_prefill_mixed_decode_gb300 import step
    q, k = torch.zeros(T, H_q, D, dtype=torch.bfloat16), torch.zeros(T, H_kv, D, dtype=torch.bfloat16)
    i = torch.zeros(T, dtype=torch.int32)
    batch = step.DeviceBatch(i[:2], i[:1], i[:1], i, i, i[:1].view(1, 1), 1, T, 0, 16, {})  # one row, one page
    pool = torch.zeros(2, H_kv, 16, D, dtype=torch.bfloat16)
    return torch, step, [q, k, k.clone(), batch], [pool, pool.clone(), torch.zeros_like(q), torch.zeros(1 << 16, dtype=torch.uint8)]


def test_step_refuses_tables_of_another_width(ms):
    """Tables that are not [max_pos, D / 2] are a mistake unless the call says that a part of the head, or none of it, turns:
    a table made for D = 64 does not turn half of every head of 128 without a word."""
    torch, step, a, b = _host_step(ms)
    tab = lambda n: torch.zeros(10, n)  # noqa: E731
    for cos, kw in ((tab(32), {}), (tab(128), {}), (None, {}), (tab(32), {"window": 16}), (None, {"window": 16}), (None, {"interleaved": True}),
                    (tab(32), {"rotary_dim": 128}), (tab(32), {"rotary_dim": 32}), (tab(64), {"rotary_dim": 64}), (tab(32), {"rotary_dim": 0}),
                    (None, {"rotary_dim": 64}), (tab(32), {"rotary_dim": 32, "interleaved": True}), (tab(128), {"interleaved": True}),
                    (tab(64).view(-1), {}), (tab(4), {"rotary_dim": 8}), (None, {"rotary_dim": -16})):
        with pytest.raises(ValueError, match="rotary_dim|must be .max_pos"):
            step.run_step(*a, cos, cos, *b, **kw)
    # what the call says and the tables bear out goes on, to the check of the device
    for cos, kw in ((tab(64), {}), (tab(32), {"rotary_dim": 64}), (tab(64), {"rotary_dim": 128}), (None, {"rotary_dim": 0}),
                    (tab(32), {"rotary_dim": 64, "interleaved": True}), (tab(32), {"interleaved": True})):
        with pytest.raises(ValueError, match="CUDA"):
            step.run_step(*a, cos, cos, *b, **kw)
    with pytest.raises(ValueError, match="q must be"):
        step.run_step(a[0].flatten(1), *a[1:], tab(64), tab(64), *b)


def test_step_refuses_bad_forms_before_it_appends(ms):
    """A window or sinks that the attention refuses leave the pools and q as they were."""
    torch, step, a, b = _host_step(ms)
    tab, seen = torch.zeros(10, 64), []
    keep, step.kv_append_rotary = step.kv_append_rotary, lambda *args, **kw: seen.append(args)
    try:
        for kw in ({"window": 0}, {"window": -3}, {"sinks": torch.zeros(3)}, {"sinks": torch.zeros(4, dtype=torch.float64)},
                   {"sinks": torch.zeros(8)[::2]}, {"window": 8, "sinks": torch.zeros(4, 1)}):
            with pytest.raises(ValueError, match="window|sinks"):
                step.run_step(*a, tab, tab, *b, **kw)
    finally:
        step.kv_append_rotary = keep
    assert not seen


def test_whole_numbers_beyond_32_bits_are_refused(ms):
    """ctypes passes a whole number's low 32 bits: the binding refuses what does not fit, where it would have taken another."""
    torch = pytest.importorskip("torch")
    for dim in (2 ** 32 + 64, 64 - 2 ** 32):
        with pytest.raises(ValueError, match="rotary_dim"):
            ms.rotary_frequencies(dim)
    for kind in ("bands", "ramp"):
        with pytest.raises(ValueError, match="original_len"):
            ms.rotary_frequencies(64, 1e4, {"kind": kind, "factor": 2.0, "original_len": 2 ** 32 + 4096, "low": 1.0, "high": 4.0})
    tab = torch.zeros(10, 16)
    for first in (2 ** 32, 2 ** 31, -2 ** 32 + 5):
        with pytest.raises(ValueError, match="first_pos"):
            ms.rotary_table_device(np.zeros(16), tab, tab.clone(), first_pos=first)
    bf, i32 = torch.bfloat16, torch.int32
    q, pool, one = torch.zeros(1, 4, 64, dtype=bf), torch.zeros(2, 2, 16, 64, dtype=bf), torch.zeros(2, dtype=i32)
    with pytest.raises(ValueError, match="window"):
        ms.mixed_step_attention_window(q, pool, pool.clone(), one, one, one, one.view(1, 2), 1, q.clone(), torch.zeros(4096, dtype=torch.uint8),
                                       16 - 2 ** 32)
    for dim in (0, -2, 3, 130, 2 ** 31 - 2):  # what fits is the C side's to refuse, and nothing is written past an array
        with pytest.raises(ms.MixedStepError):
            ms.rotary_frequencies(dim)


def test_round_driver_refuses_tables_of_another_width(ms):
    torch = pytest.importorskip("torch")
    from chunked_prefill_mixed_decode_gb300.driver import RoundDriver
    pool = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    q4 = torch.zeros(2, 2, 1152, dtype=torch.uint8)
    narrow, whole = torch.zeros(8, 16), torch.zeros(8, 32)
    for tabs, kw in ((narrow, {}), (None, {}), (narrow, {"window": 8}), (whole, {"rotary_dim": 32}), (narrow, {"rotary_dim": 64})):
        with pytest.raises(ValueError, match="rotary_dim|must be .max_pos"):
            RoundDriver(ms.Engine(2, 8), pool, pool, tabs, tabs, 4, 2, 64, **kw)
    for v, kw in ((None, {}), (pool, {"graph_buckets": [8]})):
        with pytest.raises(ValueError, match="need bf16 pools"):
            RoundDriver(ms.Engine(2, 8), q4 if v is None else pool, v, narrow, narrow, 4, 2, 64, rotary_dim=32, **kw)
