"""Python binding of libech: the MI355X (gfx950) indexer -> exact top-k ->
KV-recall path of ECHO-style lossless KV offloading.

Each function takes torch tensors (device memory, or pinned host memory for
the host pool), passes their pointers and sizes to the C ABI of the same name
(include/ech.h) and raises EchError on a non-zero return code. Nothing is
computed here; every step runs in the library's HIP kernels. Calls are
asynchronous on the given stream (default: torch's current stream).
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import torch

from . import _native
from ._native import (ECH_EARLY, ECH_FINAL, ECH_PREFILL, ECH_KEY_BF16, ECH_KEY_FP8,  # noqa: F401
                      CTR_HEAD, CTR_EPOCH, CTR_NMISS, CTR_NEVICT, CTR_RECALLED, CTR_STATUS, CTR_NWANT,
                      CTR_NPINNED, CTR_NMISS_EARLY, CTR_TICKET, CTR_NCOPIED_EARLY, CTR_LIVE,
                      CTR_NCOPIED_FINAL, CTR_FINAL_READY, CTR_FINAL_DONE, CTR_EARLY_WALK, CTR_LEN, ST_OVERFLOW, ST_BADTOK,
                      ST_BADMISS, ST_FULL, ST_TIMEOUT)

__all__ = ['ech_kv_append', 'ech_sparse_attn', 'ech_sparse_attn_ws_bytes', 'ech_index_logits', 'ech_index_logits_causal', 'ech_topk', 'ech_topk_noalloc', 'ech_topk_ws_bytes', 'ech_cache_reset',
           'ech_cache_step', 'ech_cache_step_ws_bytes', 'ech_recall', 'ech_index_logits_early',
           'ech_index_logits_early_ws_bytes', 'ech_recall_early_live', 'ech_recall_rest', 'ech_topk_early', 'ech_paged_append',
           'ech_paged_attn', 'ech_paged_attn_ws_bytes', 'ech_paged_weight', 'ech_paged_weight_ws_bytes',
           'ech_paged_evict', 'ech_paged_evict_ws_bytes', 'EchError', 'LayerState', 'lib']


class EchError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        msg = lib().ech_status_str(code).decode()
        super().__init__(f'{fn} failed: {msg} ({code})')


def lib():
    return _native.load()


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _check(fn: str, rc: int) -> None:
    if rc != 0:
        raise EchError(fn, rc)


def _key_dtype(kcache: torch.Tensor) -> int:
    if kcache.dtype in (torch.uint8, torch.float8_e4m3fn):
        return ECH_KEY_FP8
    if kcache.dtype in (torch.int16, torch.uint16, torch.bfloat16):
        return ECH_KEY_BF16
    raise TypeError(f'unsupported key dtype {kcache.dtype}')


# ------------------------------------------------------------------ stage 1
def ech_index_logits(q, w, kcache, kscale, row_tok0, row_len, max_len: int, logits, stream=None) -> None:
    """Decode indexer scores: q [R,H,D] bf16, w [R,H] f32, kcache [P,D] (uint8
    e4m3fn or bf16), kscale [P] f32 or None, row_tok0 [R] i64, row_len [R] i32,
    logits [R, ld] f32."""
    R, H, D = q.shape
    _check('ech_index_logits', lib().ech_index_logits(
        _ptr(q), _ptr(w), _ptr(kcache), _key_dtype(kcache), _ptr(kscale), _ptr(row_tok0), _ptr(row_len),
        R, H, D, int(max_len), _ptr(logits), logits.stride(0), _stream(stream)))


def ech_index_logits_causal(q, w, kcache, kscale, tok0: int, row0: int, logits, stream=None) -> None:
    """Prefill indexer scores for query rows at positions row0 .. row0+R-1 of
    the sequence starting at global token tok0 (row r sees t <= row0 + r)."""
    R, H, D = q.shape
    _check('ech_index_logits_causal', lib().ech_index_logits_causal(
        _ptr(q), _ptr(w), _ptr(kcache), _key_dtype(kcache), _ptr(kscale), int(tok0), int(row0), R, H, D,
        _ptr(logits), logits.stride(0), _stream(stream)))


# ------------------------------------------------------------------ stage 2
def ech_topk_ws_bytes(R: int, max_len: int, k: int) -> int:
    return int(lib().ech_topk_ws_bytes(R, max_len, k))


def ech_topk(logits, row_len, max_len: int, k: int, theta_in, theta_out, idx, kth, ws, stream=None) -> None:
    """Exact top-k of each row of logits [R, ld]; idx [R,k] i32 (ascending, -1
    padded), kth [R] f32, theta_in/theta_out [R] f32 or None, ws uint8."""
    R = logits.shape[0]
    _check('ech_topk', lib().ech_topk(
        _ptr(logits), logits.stride(0), _ptr(row_len), R, int(max_len), int(k), _ptr(theta_in), _ptr(theta_out),
        _ptr(idx), _ptr(kth), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


def ech_topk_noalloc(logits, row_len, max_len: int, k: int, theta_in, theta_out, idx, kth, stream=None) -> None:
    """ech_topk with the library's static per-GPU scratch array as its
    workspace (allocates nothing; calls on one GPU must not overlap)."""
    R = logits.shape[0]
    _check('ech_topk_noalloc', lib().ech_topk_noalloc(
        _ptr(logits), logits.stride(0), _ptr(row_len), R, int(max_len), int(k), _ptr(theta_in), _ptr(theta_out),
        _ptr(idx), _ptr(kth), _stream(stream)))


# ------------------------------------------------------------------ stage 3
@dataclasses.dataclass
class LayerState:
    """The fixed-size int32 tensors of one layer's slot map, on the device:
    the two maps, the epoch pins, the miss list (FINAL/PREFILL; EARLY phases
    write their own list so their rows can still be in flight while FINAL
    updates the maps) and the control counters."""
    tok2slot: torch.Tensor   # [P]
    slot2tok: torch.Tensor   # [C]
    slot_pin: torch.Tensor   # [C]
    miss: torch.Tensor       # [M_max, 2]
    ctr: torch.Tensor        # [CTR_LEN]
    miss_early: Optional[torch.Tensor] = None   # [M_early, 2]

    @property
    def P(self) -> int:
        return self.tok2slot.numel()

    @property
    def C(self) -> int:
        return self.slot2tok.numel()

    @property
    def M_max(self) -> int:
        return self.miss.shape[0]

    def miss_list(self, phase: int) -> torch.Tensor:
        return self.miss_early if phase == ECH_EARLY else self.miss

    @staticmethod
    def allocate(P: int, C: int, M_max: int, device='cuda', M_early: Optional[int] = None) -> 'LayerState':
        i32 = dict(dtype=torch.int32, device=device)
        M_early = M_max if M_early is None else M_early
        st = LayerState(torch.empty(P, **i32), torch.empty(C, **i32), torch.empty(C, **i32),
                        torch.empty((max(M_max, 1), 2), **i32), torch.empty(CTR_LEN, **i32),
                        torch.empty((max(M_early, 1), 2), **i32))
        return st


def ech_cache_reset(state: LayerState, stream=None) -> None:
    _check('ech_cache_reset', lib().ech_cache_reset(
        _ptr(state.tok2slot), state.P, _ptr(state.slot2tok), _ptr(state.slot_pin), state.C, _ptr(state.ctr),
        _stream(stream)))


def ech_cache_step_ws_bytes(phase: int, B: int, R: int, k: int, max_len: int, C: int, M_max: int) -> int:
    return int(lib().ech_cache_step_ws_bytes(phase, B, R, k, max_len, C, M_max))


def ech_cache_step(phase: int, state: LayerState, seq_tok0, seq_len, max_len: int, idx=None, k: int = 2048,
                   logits=None, theta=None, cap: int = 0, sel_slot=None, stats=None, ws=None,
                   stream=None) -> None:
    """One phase (ECH_EARLY / ECH_FINAL / ECH_PREFILL) of the slot map."""
    B = seq_tok0.shape[0]
    R = idx.shape[0] if idx is not None else B
    ld = logits.stride(0) if logits is not None else 0
    miss = state.miss_list(phase)
    _check('ech_cache_step', lib().ech_cache_step(
        phase, _ptr(state.tok2slot), state.P, _ptr(state.slot2tok), _ptr(state.slot_pin), state.C,
        _ptr(miss), miss.shape[0], _ptr(state.ctr), _ptr(seq_tok0), _ptr(seq_len), B, int(max_len),
        _ptr(idx), R, int(k), _ptr(logits), ld, _ptr(theta), int(cap), _ptr(sel_slot), _ptr(stats), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def ech_recall(host_pool, dev_cache, state: LayerState, phase: int = ECH_FINAL, stream=None) -> None:
    """Copy the rows missed by the last phase of this kind: host_pool
    [P, row_bytes] pinned (uint8/uint16), dev_cache [C, row_bytes] on the
    device."""
    row_bytes = host_pool.shape[1] * host_pool.element_size()
    miss = state.miss_list(phase)
    _check('ech_recall', lib().ech_recall(
        phase, _ptr(host_pool), host_pool.shape[0], row_bytes, _ptr(dev_cache), dev_cache.shape[0], _ptr(miss),
        _ptr(state.ctr), miss.shape[0], _stream(stream)))


# ------------------------------------------------------------------ stages 1 and 3 fused (decode, fp8 keys)
def ech_index_logits_early_ws_bytes(R: int, max_len: int, C: int, M_early: int) -> int:
    return int(lib().ech_index_logits_early_ws_bytes(R, max_len, C, M_early))


def ech_index_logits_early(q, w, kcache, kscale, row_tok0, row_len, max_len: int, logits, e0: int, e1: int, theta,
                           cap: int, state: 'LayerState', stats, ws, stream=None) -> None:
    """Decode scores of every row fused with the early fetch of sequences
    [e0, e1) (maps and early miss list, written while the scoring runs).
    ws: uint8, zero-filled before the first call."""
    R = q.shape[0]
    _check('ech_index_logits_early', lib().ech_index_logits_early(
        _ptr(q), _ptr(w), _ptr(kcache), _key_dtype(kcache), _ptr(kscale), _ptr(row_tok0), _ptr(row_len), R,
        q.shape[1], q.shape[2], int(max_len), _ptr(logits), logits.stride(0), int(e0), int(e1), _ptr(theta),
        int(cap), _ptr(state.tok2slot), state.P, _ptr(state.slot2tok), _ptr(state.slot_pin), state.C,
        _ptr(state.miss_early), state.miss_early.shape[0], _ptr(state.ctr), _ptr(stats), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))


def ech_recall_early_live(host_pool, dev_cache, state: 'LayerState', ws, stream=None, final: bool = False) -> None:
    """Copy early rows as ech_index_logits_early allocates them (enqueue on a
    second stream right after it; ech_recall(ECH_EARLY) afterwards copies the
    rest). final=True: then the rows of the FINAL phase that follows in the
    same step (state.miss), once that phase has completed its list;
    ech_recall(ECH_FINAL) afterwards copies what it left."""
    row_bytes = host_pool.shape[1] * host_pool.element_size()
    _check('ech_recall_early_live', lib().ech_recall_early_live(
        _ptr(host_pool), host_pool.shape[0], row_bytes, _ptr(dev_cache), dev_cache.shape[0], _ptr(state.miss_early),
        state.miss_early.shape[0], _ptr(state.miss) if final else None, state.miss.shape[0] if final else 0,
        _ptr(state.ctr), _ptr(ws), _stream(stream)))


def ech_topk_early(logits, row_len, max_len: int, k: int, theta_in, theta_out, idx, kth, state: 'LayerState', ws,
                   stream=None) -> None:
    """ech_topk for the rows of the last ech_index_logits_early call on ws,
    from the band lists its scoring waves wrote (theta_in: that call's)."""
    R = logits.shape[0]
    _check('ech_topk_early', lib().ech_topk_early(
        _ptr(logits), logits.stride(0), _ptr(row_len), R, int(max_len), int(k), _ptr(theta_in), _ptr(theta_out),
        _ptr(idx), _ptr(kth), _ptr(ws), ws.numel() * ws.element_size(), state.C, state.miss_early.shape[0],
        _stream(stream)))


def ech_recall_rest(host_pool, dev_cache, state: 'LayerState', stream=None) -> None:
    """What ech_recall_early_live left of the step's early and FINAL lists, in
    one launch (after the FINAL phase and the copier)."""
    row_bytes = host_pool.shape[1] * host_pool.element_size()
    _check('ech_recall_rest', lib().ech_recall_rest(
        _ptr(host_pool), host_pool.shape[0], row_bytes, _ptr(dev_cache), dev_cache.shape[0], _ptr(state.miss_early),
        state.miss_early.shape[0], _ptr(state.miss), state.miss.shape[0], _ptr(state.slot2tok), _ptr(state.ctr),
        _stream(stream)))


# ------------------------------------------------------------------ consumer
def ech_sparse_attn_ws_bytes(B: int, H: int, k: int) -> int:
    return int(lib().ech_sparse_attn_ws_bytes(B, H, k))


def ech_sparse_attn(q, dev_cache, sel_slot, sm_scale: float, out, lse=None, ws=None, stream=None) -> None:
    """Attention of each head over the rows its sequence selects: q [B, H, 576]
    bf16 bits (int16/uint16), dev_cache [C, 576] bf16 bits, sel_slot [B, k]
    int32 -> out [B, H, 512] fp32, lse [B, H] fp32 (optional)."""
    B, H = q.shape[0], q.shape[1]
    k = sel_slot.shape[1]
    _check('ech_sparse_attn', lib().ech_sparse_attn(
        _ptr(q), _ptr(dev_cache), dev_cache.shape[0], _ptr(sel_slot), B, H, k, float(sm_scale), _ptr(out),
        _ptr(lse), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))


# ------------------------------------------------------------------ growing contexts
def ech_kv_append(host_pool, kcache, kscale, state: LayerState, seq_tok0, seq_len, seq_cap, new_rows, new_keys,
                  new_scales=None, stream=None) -> None:
    """Each sequence's decoded token joins the host pool (pinned [P, row])
    and the key cache; seq_len (device int32) grows in place."""
    row_bytes = host_pool.shape[1] * host_pool.element_size()
    _check('ech_kv_append', lib().ech_kv_append(
        _ptr(host_pool), host_pool.shape[0], row_bytes, _ptr(kcache), _key_dtype(kcache), _ptr(kscale),
        _ptr(state.tok2slot), _ptr(seq_tok0), _ptr(seq_len), _ptr(seq_cap), seq_tok0.shape[0], _ptr(new_rows),
        _ptr(new_keys), _ptr(new_scales), _ptr(state.ctr), _stream(stream)))


# ------------------------------------------------------------------ resident paged cache
_BITS16 = (torch.int16, torch.uint16, torch.bfloat16)
_F32 = (torch.float32,)
_I32 = (torch.int32,)
# torch's own lookups without its wrappers' cost, where this build has them
_raw_stream = getattr(torch._C, '_cuda_getCurrentRawStream', lambda d: torch.cuda.current_stream(d).cuda_stream)
_current_device = getattr(torch._C, '_cuda_getDevice', torch.cuda.current_device)


def _arg(name: str, t: torch.Tensor, dtypes, shape, device: int, rows: bool = False) -> None:
    """Refuse a tensor that the kernels would misread: its type, shape, device,
    or strides (`rows`: only the last dimension is dense)."""
    if (t.dtype in dtypes and t.get_device() == device >= 0 and t.shape == shape
            and (t.is_contiguous() or (rows and t.stride(-1) == 1))):
        return
    if t.dtype not in dtypes:
        raise TypeError(f'{name}: unsupported dtype {t.dtype}')
    if t.shape != shape:
        raise ValueError(f'{name}: shape {tuple(t.shape)}, expected {tuple(shape)}')
    if device < 0 or t.get_device() != device:
        raise ValueError(f'{name}: on {t.device}, expected a tensor on ' + (f'GPU {device}' if device >= 0 else 'a GPU'))
    raise ValueError(f'{name}: strides {t.stride()} of shape {tuple(t.shape)} are not supported')


def _pair(name: str, t: torch.Tensor):
    """The shape of a tensor that has to have two dimensions."""
    if t.dim() != 2:
        raise ValueError(f'{name}: shape {tuple(t.shape)}, expected two dimensions')
    return t.shape


def _steps(q: torch.Tensor, T: int, H: int):
    """Values from row to row and from head to head; 0 along a dimension of one,
    whose stride says nothing."""
    return q.stride(0) if T > 1 else 0, q.stride(1) if H > 1 else 0


def _ws_arg(ws: Optional[torch.Tensor], device: int):
    """(pointer, bytes) of a workspace, or (None, 0) without one."""
    if ws is None:
        return None, 0
    if ws.get_device() != device or not ws.is_contiguous():
        raise ValueError(f'ws: expected a contiguous tensor on GPU {device}')
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _fits(*numbers: int) -> None:
    """Refuse numbers that the C ABI's 32-bit arguments would cut."""
    if max(numbers) > 0x7fffffff or min(numbers) < -0x80000000:
        raise ValueError(f'{numbers}: one of these needs more than 32 bits')


def _call(fn: str, device: int, stream, *args) -> None:
    """The library's call on the device of its tensors: on the caller's stream,
    or on that device's current one."""
    if device != _current_device():
        with torch.cuda.device(device):
            return _call(fn, device, stream, *args)
    rc = getattr(_native.load(), fn)(*args, _raw_stream(device) if stream is None else _stream(stream))
    if rc != 0:
        raise EchError(fn, rc)


def _batch_args(pool, page_table, row0, seq_len):
    """Checks shared by the paged calls; returns (device, B)."""
    dev = pool.get_device()
    B = seq_len.numel()
    _arg('seq_len', seq_len, _I32, (B,), dev)
    _arg('row0', row0, _I32, (B + 1,), dev)
    _arg('page_table', page_table, _I32, (B, _pair('page_table', page_table)[1]), dev)
    return dev, B


def ech_paged_append(pool, page_table, page_size: int, row0, seq_len, rows, status=None, stream=None) -> None:
    """A step's new rows [T, row] go into their sequences' pages: pool [slots,
    row] (any type, the type of `rows`), page_table [B, pages] i32, row0 [B+1]
    i32, seq_len [B] i32 (with the new rows), status [1] i32 or None."""
    _fits(page_size, rows.shape[0], seq_len.numel())
    dev, B = _batch_args(pool, page_table, row0, seq_len)
    n_slots, width = have = _pair('pool', pool)
    dtype = (pool.dtype,)
    _arg('pool', pool, dtype, have, dev)
    T, es = rows.shape[0], pool.element_size()
    _arg('rows', rows, dtype, (T, width), dev, rows=True)
    if status is not None:
        _arg('status', status, _I32, (1,), dev)
    _call('ech_paged_append', dev, stream, pool.data_ptr(), n_slots, width * es, page_size, page_table.data_ptr(),
          page_table.shape[1], row0.data_ptr(), seq_len.data_ptr(), B, T, rows.data_ptr(),
          (rows.stride(0) if T > 1 else width) * es, _ptr(status))


def ech_paged_attn_ws_bytes(B: int, T: int, H: int, max_rows: int, max_len: int, window: int = 0,
                            n_sink: int = 0) -> int:
    _fits(B, T, H, max_rows, max_len, window, n_sink)
    return int(lib().ech_paged_attn_ws_bytes(B, T, H, max_rows, max_len, window, n_sink))


def ech_paged_attn(q, pool, page_table, page_size: int, row0, seq_len, max_rows: int, max_len: int, sm_scale: float,
                   out, lse=None, window: int = 0, n_sink: int = 0, ws=None, stream=None) -> None:
    """Causal attention of a step's new rows over their sequences' pages, with
    an optional sliding window and n_sink first tokens that stay visible: q
    [T, H, 576] bf16 (or its bits; rows and heads may be strided), pool [slots,
    576] bf16 -> out [T, H, 512] bf16, lse [T, H] fp32 (optional)."""
    _fits(page_size, max_rows, max_len, window, n_sink, q.shape[0], seq_len.numel())
    _arg('pool', pool, _BITS16, (pool.shape[0], 576), pool.get_device())
    dev, B = _batch_args(pool, page_table, row0, seq_len)
    T, H = q.shape[0], q.shape[1] if q.dim() == 3 else -1
    _arg('q', q, _BITS16, (T, H, 576), dev, rows=True)
    _arg('out', out, _BITS16, (T, H, 512), dev)
    if lse is not None:
        _arg('lse', lse, _F32, (T, H), dev)
    wp, wb = _ws_arg(ws, dev)
    _call('ech_paged_attn', dev, stream, q.data_ptr(), *_steps(q, T, H), pool.data_ptr(), pool.shape[0],
          page_size, page_table.data_ptr(), page_table.shape[1], row0.data_ptr(), seq_len.data_ptr(), B, T, H, max_rows,
          max_len, window, n_sink, sm_scale, out.data_ptr(), _ptr(lse), wp, wb)


def ech_paged_weight_ws_bytes(B: int, T: int, H: int, max_rows: int, max_len: int) -> int:
    _fits(B, T, H, max_rows, max_len)
    return int(lib().ech_paged_weight_ws_bytes(B, T, H, max_rows, max_len))


def ech_paged_weight(q, lse, pool, page_table, page_size: int, row0, seq_len, max_rows: int, max_len: int,
                     sm_scale: float, acc_in, acc_out, decay: float = 1.0, window: int = 0, n_sink: int = 0, ws=None,
                     stream=None) -> None:
    """The attention weight each cached token received from the step's rows
    and heads (lse: that of ech_paged_attn), added to decay * acc_in: acc_in
    [B, >= max_len] fp32 or None, acc_out like it (may be acc_in)."""
    _fits(page_size, max_rows, max_len, window, n_sink, q.shape[0], seq_len.numel())
    _arg('pool', pool, _BITS16, (pool.shape[0], 576), pool.get_device())
    dev, B = _batch_args(pool, page_table, row0, seq_len)
    T, H = q.shape[0], q.shape[1] if q.dim() == 3 else -1
    _arg('q', q, _BITS16, (T, H, 576), dev, rows=True)
    _arg('lse', lse, _F32, (T, H), dev)
    ld = _pair('acc_out', acc_out)[1]
    _arg('acc_out', acc_out, _F32, (B, ld), dev)
    if acc_in is not None:
        _arg('acc_in', acc_in, _F32, (B, ld), dev)
    wp, wb = _ws_arg(ws, dev)
    _call('ech_paged_weight', dev, stream, q.data_ptr(), *_steps(q, T, H), lse.data_ptr(), pool.data_ptr(),
          pool.shape[0], page_size, page_table.data_ptr(), page_table.shape[1], row0.data_ptr(), seq_len.data_ptr(), B,
          T, H, max_rows, max_len, window, n_sink, sm_scale, _ptr(acc_in), acc_out.data_ptr(), ld, decay, wp, wb)


def ech_paged_evict_ws_bytes(B: int, max_len: int, keep: int) -> int:
    _fits(B, max_len, keep)
    return int(lib().ech_paged_evict_ws_bytes(B, max_len, keep))


def ech_paged_evict(acc, seq_len, max_len: int, keep: int, n_sink: int, n_recent: int, kept, len_out, acc_out=None,
                    pool=None, src_table=None, dst_table=None, page_size: int = 1, ws=None, stream=None) -> None:
    """Keep `keep` tokens of each longer sequence: the first n_sink, the last
    n_recent and the heaviest between (acc [B, >= max_len] fp32). kept [B,
    keep] i32 (ascending, -1 padded), len_out [B] i32, acc_out like acc or
    None. With a pool the kept rows move from src_table's pages to dst_table's
    (src_table itself: compacted in place)."""
    dev, B = acc.get_device(), seq_len.numel()
    _fits(B, max_len, keep, n_sink, n_recent, page_size)
    _arg('seq_len', seq_len, _I32, (B,), dev)
    ld = _pair('acc', acc)[1]
    _arg('acc', acc, _F32, (B, ld), dev)
    _arg('kept', kept, _I32, (B, keep), dev)
    _arg('len_out', len_out, _I32, (B,), dev)
    if acc_out is not None:
        _arg('acc_out', acc_out, _F32, (B, ld), dev)
    n_slots = row_bytes = pt_ld = 0
    if pool is not None:
        _arg('pool', pool, (pool.dtype,), _pair('pool', pool), dev)
        if src_table is None or dst_table is None:
            raise ValueError('src_table and dst_table are needed to move the rows of a pool')
        pt_ld = _pair('src_table', src_table)[1]
        _arg('src_table', src_table, _I32, (B, pt_ld), dev)
        _arg('dst_table', dst_table, _I32, (B, pt_ld), dev)
        n_slots, row_bytes = pool.shape[0], pool.shape[1] * pool.element_size()
    wp, wb = _ws_arg(ws, dev)
    _call('ech_paged_evict', dev, stream, acc.data_ptr(), ld, seq_len.data_ptr(), B, max_len, keep, n_sink, n_recent,
          kept.data_ptr(), _ptr(acc_out), len_out.data_ptr(), _ptr(pool), n_slots, row_bytes, page_size,
          _ptr(src_table) if pool is not None else None, _ptr(dst_table) if pool is not None else None, pt_ld, wp, wb)
