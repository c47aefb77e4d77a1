"""One mixed step end to end through the C ABI: host metadata -> device, append, attention.

Marshalling only (torch for device memory and streams): the packing runs in
ms_build_batch_metadata, the arithmetic in ms_kv_append_rope and
ms_mixed_step_attention.
"""
from __future__ import annotations

import dataclasses

import numpy as np

from . import (attention_workspace_size, build_batch_metadata_device, check_sinks, kv_append_rope_q4, kv_append_rotary,
               mixed_step, mixed_step_attention, mixed_step_attention_q4, mixed_step_attention_ragged, mixed_step_attention_window,
               mixed_step_cross_attention, q4_block_bytes, rope_table, rotary_frequencies, rotary_table_device)

META_KEYS = ("cu_seqlens_q", "q_start_pos", "context_lens", "positions", "slot_mapping", "block_tables")
RAGGED_KEYS = ("cu_seqlens_q", "q_start_pos", "context_lens", "positions", "slot_mapping", "bt_offsets", "bt_pages")


def _keys(meta: dict):
    return RAGGED_KEYS if "bt_offsets" in meta else META_KEYS


@dataclasses.dataclass
class DeviceBatch:
    """Device copies of one step's metadata plus the host-side sizes the calls need."""
    cu_seqlens_q: object
    q_start_pos: object
    context_lens: object
    positions: object
    slot_mapping: object
    block_tables: object
    num_rows: int
    num_tokens: int
    num_decodes: int
    context_total: int
    host: dict  # the metadata's host arrays (empty for a batch built on the GPU)
    bt_offsets: object = None  # ragged block table (then block_tables holds the pages back to back)

    @property
    def ragged(self) -> bool:
        return self.bt_offsets is not None

    @property
    def h2d_bytes(self) -> int:
        return sum(int(np.asarray(self.host[k]).nbytes) for k in _keys(self.host) if k in self.host)


def to_device(meta: dict, device, non_blocking: bool = False) -> DeviceBatch:
    import torch
    t = {}
    for k in _keys(meta):
        a = np.ascontiguousarray(meta[k], dtype=np.int32)
        if a.size == 0:
            a = np.zeros(1, dtype=np.int32)  # keep a valid device pointer for empty arrays
        src = torch.from_numpy(a)
        if non_blocking:
            src = src.pin_memory()
        t[k] = src.to(device, non_blocking=non_blocking)
    S = int(meta["num_rows"])
    ctx_total = int(np.asarray(meta["context_lens"], dtype=np.int64).sum())
    if "bt_offsets" in meta:
        return DeviceBatch(t["cu_seqlens_q"], t["q_start_pos"], t["context_lens"], t["positions"],
                           t["slot_mapping"], t["bt_pages"], S, int(meta["num_tokens"]), int(meta["num_decodes"]),
                           ctx_total, meta, bt_offsets=t["bt_offsets"])
    bt = t["block_tables"]
    stride = int(meta["bt_stride"])
    t["block_tables"] = bt.view(max(S, 1), max(stride, 1)) if S > 0 and stride > 0 else bt.view(1, 1)
    return DeviceBatch(t["cu_seqlens_q"], t["q_start_pos"], t["context_lens"], t["positions"], t["slot_mapping"],
                       t["block_tables"], S, int(meta["num_tokens"]), int(meta["num_decodes"]), ctx_total, meta)


class MetaStager:
    """Reusable pinned staging for one step's metadata: the six arrays are packed
    into one pinned host buffer and reach the device in a single copy.

    Two host/device buffer pairs alternate; a host buffer is refilled only after
    the copy that last read it has finished (an event per buffer).  Device
    buffers are reused in stream order, so the kernels of a step finish reading
    one before a later copy on the same stream overwrites it.
    """

    def __init__(self, max_rows: int, max_tokens: int, max_bt: int, device):
        self.device = device
        self.cap = 0
        self.events = [None, None]
        self.flip = 0
        self._grow(3 * max_rows + 1 + 2 * max_tokens + max_bt + 6 * 4)  # plus alignment slack

    def _grow(self, cap: int):
        import torch
        for ev in self.events:
            if ev is not None:
                ev.synchronize()
        torch.cuda.synchronize(self.device)  # earlier steps may still read the old device buffers
        self.cap = cap
        self.host = [torch.empty(cap, dtype=torch.int32).pin_memory() for _ in range(2)]
        self.dev = [torch.empty(cap, dtype=torch.int32, device=self.device) for _ in range(2)]
        self.events = [None, None]

    def stage(self, meta: dict, stream=None) -> DeviceBatch:
        import torch
        S, T, stride = int(meta["num_rows"]), int(meta["num_tokens"]), int(meta["bt_stride"])
        ragged = "bt_offsets" in meta
        n_bt = (S + 1 + int(meta["bt_offsets"][S])) if ragged else S * stride
        need = 3 * S + 1 + 2 * T + n_bt + 7 * 4
        if need > self.cap:
            self._grow(max(need, 2 * self.cap))
        i = self.flip
        self.flip ^= 1
        if self.events[i] is not None:
            self.events[i].synchronize()
        hv = self.host[i].numpy()
        views, off = {}, 0
        tabs = ((("bt_offsets", S + 1), ("bt_pages", int(meta["bt_offsets"][S]))) if ragged
                else (("block_tables", S * stride),))
        for k, n in (("cu_seqlens_q", S + 1), ("q_start_pos", S), ("context_lens", S), ("positions", T),
                     ("slot_mapping", T)) + tabs:
            n_alloc = max(n, 1)
            if off + n_alloc > self.cap:
                raise ValueError("metadata larger than the stager's capacity")
            hv[off:off + n] = np.asarray(meta[k], dtype=np.int32).reshape(-1)[:n]
            views[k] = (off, n_alloc)
            off += (n_alloc + 3) & ~3  # keep each array 16-byte aligned
        st = stream if stream is not None else torch.cuda.current_stream(self.dev[i].device)
        with torch.cuda.stream(st):
            self.dev[i][:off].copy_(self.host[i][:off], non_blocking=True)
            ev = torch.cuda.Event()
            ev.record(st)
        self.events[i] = ev
        d = {k: self.dev[i][o:o + n] for k, (o, n) in views.items()}
        ctx_total = int(np.asarray(meta["context_lens"], dtype=np.int64).sum())
        if ragged:
            return DeviceBatch(d["cu_seqlens_q"], d["q_start_pos"], d["context_lens"], d["positions"],
                               d["slot_mapping"], d["bt_pages"], S, T, int(meta["num_decodes"]), ctx_total, meta,
                               bt_offsets=d["bt_offsets"])
        bt = d["block_tables"].view(S, stride) if S > 0 and stride > 0 else d["block_tables"][:1].view(1, 1)
        return DeviceBatch(d["cu_seqlens_q"], d["q_start_pos"], d["context_lens"], d["positions"],
                           d["slot_mapping"], bt, S, T, int(meta["num_decodes"]), ctx_total, meta)


def rope_tables_device(max_pos: int, D: int, device, base: float = 10000.0):
    import torch
    cos, sin = rope_table(max_pos, D, base)
    return torch.from_numpy(cos).to(device), torch.from_numpy(sin).to(device)


def rotary_tables(max_pos: int, rotary_dim: int, device, base: float = 10000.0, scaling: dict = None, first_pos: int = 0):
    """Cosines and sines [max_pos, rotary_dim / 2] of the positions from ``first_pos`` on, made on the GPU, with the
    frequencies scaled as ``scaling`` says (rotary_frequencies)."""
    import torch
    freq, amplitude = rotary_frequencies(rotary_dim, base, scaling)
    cos, sin = (torch.empty((max_pos, rotary_dim // 2), dtype=torch.float32, device=device) for _ in range(2))
    with torch.cuda.device(cos.device):
        rotary_table_device(freq, cos, sin, amplitude=amplitude, first_pos=first_pos)
    return cos, sin


def workspace_for(batch: DeviceBatch, H_q: int, H_kv: int, D: int, device, q4: bool = False):
    """A zeroed workspace for the attention of this batch; ``q4``: with the room that a step over a 4-bit pool, a window
    or an encoder's states uses to cut few long chunk items into parts (it runs without, on whole items)."""
    import torch
    n = attention_workspace_size(max(batch.num_rows, 1), max(batch.num_tokens, 1), batch.context_total, H_q, H_kv,
                                 D, q4=q4)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=device)


def kv_pool_q4(num_pages: int, H_kv: int, D: int, device):
    """A 4-bit K/V pool of zeros: one uint8 tensor [num_pages, H_kv, q4_block_bytes(D)] in place of a K and a V pool."""
    import torch
    return torch.zeros((num_pages, H_kv, q4_block_bytes(D)), dtype=torch.uint8, device=device)


class StepTables:
    """A step's metadata built on the GPU from the requests' lengths, into buffers of fixed sizes.

    ``page_tables`` [rows, stride] (device int32) are the requests' pages.  With ``free_pages`` (device int32, all of
    them free at the start) a request holds exactly the pages of its cached tokens and ``build`` takes those that it
    lacks from the end of the list; without, the tables already hold every page.  ``build`` enqueues one kernel and
    returns a DeviceBatch over the buffers: ``max_tokens`` tokens (the ones past the step's own are pad tokens), and
    ``max_context`` for the sum of the contexts, by default the whole pool (requests that share pages may need more).
    Nothing in it depends on host data, so a step can be captured and replayed while ``cached_lens`` and ``new_tokens``
    change on the GPU.  ``info`` [4] and ``status`` [1] are those of
    build_batch_metadata_device.

    The first ``free_state[0]`` entries of ``free_pages`` are the free ones.  Pages that a finished request held go back
    between two builds by writing them behind those and adding to the count, on the GPU too: ``free_pages[n:n + k] =
    pages; free_state[0] += k``.
    """

    def __init__(self, page_tables, num_pages: int, max_tokens: int, free_pages=None, max_context: int = None):
        import torch
        rows, stride = page_tables.shape
        dev = page_tables.device

        def buf(*shape):
            return torch.zeros(shape, dtype=torch.int32, device=dev)
        self.page_tables, self.num_pages, self.free_pages = page_tables, int(num_pages), free_pages
        self.cu_seqlens_q, self.q_start_pos, self.context_lens = buf(rows + 1), buf(rows), buf(rows)
        self.positions, self.slot_mapping = buf(max_tokens), buf(max_tokens)
        self.block_tables, self.info, self.status = buf(rows, stride), buf(4), buf(1)
        self.free_state = None
        if free_pages is not None:
            self.free_state = torch.tensor([free_pages.numel(), 0], dtype=torch.int32, device=dev)
        self.batch = DeviceBatch(self.cu_seqlens_q, self.q_start_pos, self.context_lens, self.positions,
                                 self.slot_mapping, self.block_tables, rows, int(max_tokens), 0,
                                 16 * self.num_pages if max_context is None else int(max_context), {})

    def build(self, cached_lens, new_tokens, stream=None) -> DeviceBatch:
        free = {}
        if self.free_pages is not None:
            free = {"free_pages": self.free_pages, "free_count": self.free_state[:1], "free_state": self.free_state}
        build_batch_metadata_device(cached_lens, new_tokens, self.page_tables, self.num_pages, self.cu_seqlens_q,
                                    self.q_start_pos, self.context_lens, self.positions, self.slot_mapping,
                                    block_tables=self.block_tables, info=self.info, dev_status=self.status,
                                    stream=stream, **free)
        return self.batch


def check_rotary_tables(cos, sin, D: int, rotary_dim: int = None, interleaved: bool = False) -> None:
    """The tables of a step are [max_pos, rotary_dim / 2], or None for a ``rotary_dim`` of 0 (nothing turns).  Without
    ``rotary_dim`` the whole head turns, D elements; in ``interleaved`` pairs as many as the tables have."""
    if rotary_dim is not None and (rotary_dim % 16 != 0 or not 0 <= rotary_dim <= D):
        raise ValueError(f"rotary_dim must be a multiple of 16 from 0 to {D}, got {rotary_dim}")
    if cos is None or sin is None:
        if cos is not sin or rotary_dim != 0:
            raise ValueError("cos and sin are required, both of them, unless rotary_dim is 0")
        return
    if cos.dim() != 2:
        raise ValueError("cos must be [max_pos, rotary_dim/2]")
    R = (min(2 * cos.shape[1], D) if interleaved else D) if rotary_dim is None else rotary_dim
    if 2 * cos.shape[1] != R or R == 0:
        raise ValueError(f"cos must be [max_pos, {R // 2}] for {R} of {D} elements that turn (rotary_dim), got {tuple(cos.shape)}")


def run_step(q, k, v, batch: DeviceBatch, cos, sin, k_cache, v_cache, out, workspace, q_rot=None,
             dev_status=None, scale=None, stream=None, interleaved: bool = False, window: int = None, sinks=None,
             rotary_dim: int = None):
    """One step of one layer; returns q_rot.

    Where the whole head turns in halves and every token sees all keys up to its own this is ms_mixed_step (the append,
    then the attention, with the prologue inside the append's launch on small steps).  With a ``rotary_dim`` of less than
    the head (0, with tables of None: nothing turns), ``interleaved`` pairs, or q, k, v whose tokens' rows lie apart, the
    append is kv_append_rotary; with a ``window`` or ``sinks`` the attention is mixed_step_attention_window.  Tables of
    another width than ``rotary_dim`` says (check_rotary_tables) are refused.  The append and the attention are then two
    calls: what the attention alone refuses (a workspace too small, a count of heads) is refused behind the append."""
    if q.dim() != 3:
        raise ValueError(f"q must be [T, H_q, D], got {tuple(q.shape)}")
    if q_rot is None:
        q_rot = q
    T, D = batch.num_tokens, q.shape[2]
    check_rotary_tables(cos, sin, D, rotary_dim, interleaved)
    if window is not None and window < 1:  # here, and the sinks too: ahead of the append, which changes the pools
        raise ValueError(f"window must be at least 1, got {window}")
    check_sinks(sinks, q.shape[1])
    rows = (q[:T], k[:T], v[:T])
    if interleaved or cos is None or 2 * cos.shape[1] != D or not all(x.is_contiguous() for x in rows):
        kv_append_rotary(*rows, batch.positions, batch.slot_mapping, cos, sin, k_cache, v_cache, q_rot=q_rot[:T],
                         interleaved=interleaved, dev_status=dev_status, stream=stream)
    elif window is None and sinks is None:
        mixed_step(*rows, batch.positions, batch.slot_mapping, cos, sin, k_cache, v_cache, q_rot[:T], batch.cu_seqlens_q,
                   batch.q_start_pos, batch.context_lens, batch.block_tables, batch.context_total, out[:T], workspace,
                   bt_offsets=batch.bt_offsets if batch.ragged else None, dev_status=dev_status, scale=scale,
                   stream=stream)
        return q_rot
    else:
        kv_append_rotary(*rows, batch.positions, batch.slot_mapping, cos, sin, k_cache, v_cache, q_rot=q_rot[:T],
                         dev_status=dev_status, stream=stream)
    attend(q_rot[:T], k_cache, v_cache, batch, out[:T], workspace, scale=scale, stream=stream, window=window, sinks=sinks)
    return q_rot


def attend(q_rot, k_cache, v_cache, batch: DeviceBatch, out, workspace, scale=None, stream=None, window: int = None,
           sinks=None) -> None:
    """The attention call of a staged batch, with its padded or ragged block table; with a ``window`` or ``sinks`` over
    the last ``window`` keys (all of them where it is None)."""
    if window is not None or sinks is not None:
        mixed_step_attention_window(q_rot, k_cache, v_cache, batch.cu_seqlens_q, batch.q_start_pos, batch.context_lens,
                                    batch.block_tables, batch.context_total, out, workspace,
                                    2 ** 31 - 1 if window is None else window, sinks=sinks,
                                    bt_offsets=batch.bt_offsets if batch.ragged else None, scale=scale, stream=stream)
    elif batch.ragged:
        mixed_step_attention_ragged(q_rot, k_cache, v_cache, batch.cu_seqlens_q, batch.q_start_pos,
                                    batch.context_lens, batch.bt_offsets, batch.block_tables, batch.context_total,
                                    out, workspace, scale=scale, stream=stream)
    else:
        mixed_step_attention(q_rot, k_cache, v_cache, batch.cu_seqlens_q, batch.q_start_pos, batch.context_lens,
                             batch.block_tables, batch.context_total, out, workspace, scale=scale, stream=stream)


def append_states(k, v, slot_mapping, k_cache, v_cache, dev_status=None, stream=None) -> None:
    """An encoder's keys and values [n, H_kv, D] into the pages of their pools, as they are."""
    kv_append_rotary(None, k, v, None, slot_mapping, None, None, k_cache, v_cache, dev_status=dev_status, stream=stream)


def cross_attend(q, k_cache, v_cache, batch: DeviceBatch, key_lens, block_tables, key_total: int, out, workspace,
                 bt_offsets=None, scale=None, stream=None) -> None:
    """The batch's tokens over the states of their rows' encoders: row s sees the ``key_lens[s]`` keys that row s of
    ``block_tables`` (or of the ragged list with ``bt_offsets``) names, in pools of their own.  ``workspace`` may be the
    one of the step's self-attention where it is large enough (attention_workspace_size with ``key_total`` for the
    contexts' sum)."""
    T = batch.num_tokens
    mixed_step_cross_attention(q[:T], k_cache, v_cache, batch.cu_seqlens_q, key_lens, block_tables, key_total, out[:T],
                               workspace, bt_offsets=bt_offsets, scale=scale, stream=stream)


def run_step_q4(q, k, v, batch: DeviceBatch, cos, sin, kv_cache, out, workspace, q_rot=None, dev_status=None,
                scale=None, stream=None):
    """run_step over a 4-bit pool: the append, then the attention; returns q_rot."""
    if q_rot is None:
        q_rot = q
    T = batch.num_tokens
    kv_append_rope_q4(q[:T], k[:T], v[:T], batch.positions, batch.slot_mapping, cos, sin, kv_cache, q_rot=q_rot[:T],
                      dev_status=dev_status, stream=stream)
    mixed_step_attention_q4(q_rot[:T], kv_cache, batch.cu_seqlens_q, batch.q_start_pos, batch.context_lens,
                            batch.block_tables, batch.context_total, out[:T], workspace,
                            bt_offsets=batch.bt_offsets if batch.ragged else None, scale=scale, stream=stream)
    return q_rot
