"""Torch-facing calls of the operators around the selected-slot attention
(include/qsa_layer.h): the per-head norm and rotation that fills the cache, the index keys
of the cheap score, the selection of slots, and the attention of one new token over the
paged cache.  Like the rest of the package it turns tensors into pointers and computes
nothing; work is enqueued on ``stream`` (default: torch's current stream) and nothing is
synchronised.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools

import torch

from ._binding import QSA_OK, QSAError, load_library, qsa_last_error_detail

_E4M3 = torch.float8_e4m3fn


def _check(name, t, dtype, device, shape=None):
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dim() > 0 and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")


def _check_err_word(t, device):
    if t.device != device or t.element_size() != 4:
        raise ValueError(f"err_word must be a 4-byte integer tensor on {device}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _cuda_device(name, t):
    if t.device.type != "cuda":
        raise ValueError(f"{name} runs on CUDA tensors only")
    return t.device


def _on(device, stream):
    """Makes `device`, and `stream` when one is given, current: buffers allocated inside
    then belong to the stream that uses them."""
    if stream is not None:
        return torch.cuda.stream(stream)
    if torch.cuda.current_device() != device.index:
        return torch.cuda.device(device)
    return contextlib.nullcontext()


def _raise(status):
    raise QSAError(status, qsa_last_error_detail())


@functools.lru_cache(maxsize=None)
def _sm_count(index):
    return torch.cuda.get_device_properties(index).multi_processor_count


def qk_norm_rope(q, positions, inv_freq, k=None, v=None, q_weight=None, k_weight=None, eps=1e-6,
                 weight_offset=0.0, sections=None, interleaved=False, rope_scale=1.0, q_out=None,
                 k_cache=None, v_cache=None, slots=None, k_scale=1.0, v_scale=1.0, err_word=None,
                 stream=None):
    """Per-head RMS norm and position rotation of queries and keys in one pass, with keys and
    values stored to their cache slots.

    q [T, Hq, D], k / v [T, Hkv, D] bf16 (D 64, 128 or 256; v is only stored); q_weight /
    k_weight bf16 [D], or None for no norm (weight_offset is added to them); positions int32
    [T], or [axes, T] with ``sections``: how many of the rotated pairs each axis turns;
    inv_freq float32 [rot / 2].  Pairs are (i, i + rot / 2), or (2 i, 2 i + 1) with
    ``interleaved``.  Row t of k and v goes to row slots[t] (int32, -1 = not stored) of
    k_cache / v_cache [S, Hkv, D], bf16 or float8_e4m3fn (then divided by k_scale / v_scale
    and saturated).  Without k_cache the rotated keys come back as a new tensor.  q_out may
    be q.  Returns (q_out, rotated keys or None).
    """
    device = _cuda_device("qk_norm_rope", q)
    T, Hq, D = q.shape
    _check("q", q, torch.bfloat16, device)
    rot = 2 * inv_freq.shape[0]
    _check("inv_freq", inv_freq, torch.float32, device, (rot // 2,))
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    _check("positions", positions, torch.int32, device, (T,) if positions.dim() == 1 else (axes, T))
    if sections is None and axes != 1:
        raise ValueError("positions of several axes need sections")
    if sections is not None and len(sections) != axes:
        raise ValueError("one section per axis of positions")
    Hkv = 0
    if k is not None:
        Hkv = k.shape[1]
        _check("k", k, torch.bfloat16, device, (T, Hkv, D))
    elif v is not None or k_cache is not None or v_cache is not None:
        raise ValueError("v, k_cache and v_cache need k")
    if v is not None:
        _check("v", v, torch.bfloat16, device, (T, Hkv, D))
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _check(name, w, torch.bfloat16, device, (D,))
    fp8 = k_cache is not None and k_cache.dtype == _E4M3
    rows = T
    if k_cache is not None:
        rows = k_cache.shape[0]
        _check("k_cache", k_cache, _E4M3 if fp8 else torch.bfloat16, device, (rows, Hkv, D))
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache come together")
    if v_cache is not None:
        if k_cache is None:
            raise ValueError("v_cache needs k_cache")
        _check("v_cache", v_cache, k_cache.dtype, device, (rows, Hkv, D))
    if slots is not None:
        if k_cache is None:
            raise ValueError("slots need k_cache")
        _check("slots", slots, torch.int32, device, (T,))
    if err_word is not None:
        _check_err_word(err_word, device)
    with _on(device, stream):
        if q_out is None:
            q_out = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=device)
        else:
            _check("q_out", q_out, torch.bfloat16, device, (T, Hq, D))
        k_out = None
        if k is not None and k_cache is None:
            k_out = torch.empty(T, Hkv, D, dtype=torch.bfloat16, device=device)
        k_dst = k_cache if k_cache is not None else k_out
        st = load_library().qsa_qk_norm_rope(
            q.data_ptr(), q.stride(0), q.stride(1),
            *((k.data_ptr(), k.stride(0), k.stride(1)) if k is not None else (None, 0, 0)),
            *((v.data_ptr(), v.stride(0), v.stride(1)) if v is not None else (None, 0, 0)),
            _ptr(q_weight), _ptr(k_weight), weight_offset, eps, positions.data_ptr(),
            positions.stride(0) if axes > 1 else 0, inv_freq.data_ptr(), rot,
            1 if interleaved else 0,
            None if sections is None else (ctypes.c_int32 * axes)(*sections), axes, rope_scale, T,
            Hq, Hkv, D, q_out.data_ptr(), q_out.stride(0), q_out.stride(1),
            *((k_dst.data_ptr(), k_dst.stride(0), k_dst.stride(1)) if k_dst is not None else (None, 0, 0)),
            *((v_cache.data_ptr(), v_cache.stride(0), v_cache.stride(1)) if v_cache is not None
              else (None, 0, 0)),
            _ptr(slots), rows, 1 if fp8 else 0, k_scale, v_scale, _ptr(err_word),
            torch.cuda.current_stream(device).cuda_stream)
    if st != QSA_OK:
        _raise(st)
    return q_out, k_out


def pack_index_keys(keys, blocks, codes, scales, block=4, err_word=None, stream=None):
    """int8 codes and scales of the cheap score's keys, one per named micro-block.

    keys bf16 [S, Di]: one index key per cache slot; blocks int32 [n]: physical micro-blocks
    (slot // block; -1 is skipped); codes int8 [S // block, Di] and scales float32
    [S // block] are written in place for the named blocks.  Returns (codes, scales).
    """
    device = _cuda_device("pack_index_keys", keys)
    S, Di = keys.shape
    if block < 1:
        raise ValueError("block must be positive")
    _check("keys", keys, torch.bfloat16, device)
    _check("blocks", blocks, torch.int32, device, (blocks.numel(),))
    _check("codes", codes, torch.int8, device, (S // block, Di))
    _check("scales", scales, torch.float32, device, (S // block,))
    if err_word is not None:
        _check_err_word(err_word, device)
    with _on(device, stream):
        st = load_library().qsa_pack_index_keys(
            keys.data_ptr(), keys.stride(0), blocks.data_ptr(), blocks.numel(), block, Di, S,
            codes.data_ptr(), codes.stride(0), scales.data_ptr(), _ptr(err_word),
            torch.cuda.current_stream(device).cuda_stream)
    if st != QSA_OK:
        _raise(st)
    return codes, scales


def qsa_select_slots_workspace_bytes(Tq, B, P, page_size, Hi, Di, block) -> int:
    """Workspace bytes of qsa_select_slots; raises QSAError for invalid sizes."""
    n = int(load_library().qsa_select_slots_workspace_bytes(Tq, B, P, page_size, Hi, Di, block))
    if n == ctypes.c_size_t(-1).value:
        raise QSAError(1, qsa_last_error_detail())
    return n


def select_slots(q, weight, codes, scales, page_table, seq_lens, top_blocks, page_size, block=4,
                 cu_q=None, sink_blocks=0, local_blocks=0, slot_idx=None, width=None,
                 workspace=None, err_word=None, stream=None):
    """The slots that each query row attends to, by a cheap score of its sequence's
    micro-blocks: (slot_idx int32 [Tq, top_blocks * block + block - 1], width int32 [Tq]), as
    sparse_prefill takes them.

    q bf16 [Tq, Hi, Di] and weight float32 [Tq, Hi] of the score's heads; codes int8
    [pages * page_size // block, Di] and scales from pack_index_keys; page_table int32
    [B, P], seq_lens int32 [B] tokens of each sequence, the rows' own included; cu_q int32
    [B + 1]: the rows of sequence b are cu_q[b] .. cu_q[b + 1] - 1 (non-decreasing), its last
    tokens (None: one row per sequence).  A row takes the top_blocks complete blocks of the
    largest score among those it sees (the first sink_blocks and the last local_blocks
    always; ties to the lower block), in ascending order, then the slots of the incomplete
    block at its end; -1 fills the rest.  Rows of no sequence are left as they are.
    """
    device = _cuda_device("select_slots", q)
    Tq, Hi, Di = q.shape
    _check("q", q, torch.bfloat16, device)
    _check("weight", weight, torch.float32, device, (Tq, Hi))
    _check("codes", codes, torch.int8, device)
    if codes.dim() != 2 or codes.shape[1] != Di:
        raise ValueError("codes must be [blocks, Di]")
    _check("scales", scales, torch.float32, device, (codes.shape[0],))
    _check("page_table", page_table, torch.int32, device)
    if page_table.dim() != 2:
        raise ValueError("page_table must be [B, P]")
    B, P = page_table.shape
    _check("seq_lens", seq_lens, torch.int32, device, (B,))
    if cu_q is not None:
        _check("cu_q", cu_q, torch.int32, device, (B + 1,))
    if err_word is not None:
        _check_err_word(err_word, device)
    if block < 1 or page_size < 1 or page_size % block:
        raise ValueError("page_size must be a positive multiple of block")
    need = qsa_select_slots_workspace_bytes(Tq, B, P, page_size, Hi, Di, block)
    with _on(device, stream):
        if slot_idx is None:
            slot_idx = torch.empty(Tq, max(top_blocks, 0) * block + block - 1, dtype=torch.int32, device=device)
        else:
            _check("slot_idx", slot_idx, torch.int32, device, (Tq, top_blocks * block + block - 1))
        if width is None:
            width = torch.empty(Tq, dtype=torch.int32, device=device)
        else:
            _check("width", width, torch.int32, device, (Tq,))
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            _check("workspace", workspace, torch.uint8, device)
        st = load_library().qsa_select_slots(
            q.data_ptr(), q.stride(0), q.stride(1), weight.data_ptr(), weight.stride(0),
            codes.data_ptr(), codes.stride(0), scales.data_ptr(), page_table.data_ptr(),
            page_table.stride(0), seq_lens.data_ptr(), _ptr(cu_q), Tq, B, P,
            codes.shape[0] // (page_size // block), page_size, Hi, Di, block, top_blocks,
            sink_blocks, local_blocks, slot_idx.data_ptr(), slot_idx.stride(0), width.data_ptr(),
            workspace.data_ptr(), workspace.numel(), _ptr(err_word),
            torch.cuda.current_stream(device).cuda_stream)
    if st != QSA_OK:
        _raise(st)
    return slot_idx, width


def qsa_paged_decode_plan(B, Hq, Hkv, D, P, page_size, num_sms, nsplit_request=0):
    """(nsplit, workspace_bytes) for this shape; raises QSAError for invalid shapes."""
    ws = ctypes.c_size_t(0)
    n = int(load_library().qsa_paged_decode_plan(B, Hq, Hkv, D, P, page_size, num_sms,
                                                 nsplit_request, ctypes.byref(ws)))
    if n < 0:
        raise QSAError(-n, qsa_last_error_detail())
    return n, int(ws.value)


def paged_decode(q, k_cache, v_cache, page_table, seq_lens, page_size, scale=None, k_scale=1.0,
                 v_scale=1.0, out=None, lse=None, nsplit=0, workspace=None, err_word=None,
                 stream=None):
    """Attention of one new token per sequence over its whole paged cache.

    q [B, Hq, 256] bf16; k_cache / v_cache [S, Hkv, 256] bf16 or float8_e4m3fn (dequantised
    as code * k_scale, v_scale); page_table int32 [B, P]: token i of sequence b lies in slot
    page_table[b, i // page_size] * page_size + i % page_size; seq_lens int32 [B]; scale
    defaults to 1/16.  Returns out [B, Hq, 256] bf16 (zeros for an empty sequence); lse
    (float32 [B, Hq], optional) receives the base-2 log-sum-exp of the scaled scores.
    """
    device = _cuda_device("paged_decode", q)
    B, Hq, D = q.shape
    S, Hkv, _ = k_cache.shape
    fp8 = k_cache.dtype == _E4M3
    _check("q", q, torch.bfloat16, device)
    _check("k_cache", k_cache, _E4M3 if fp8 else torch.bfloat16, device, (S, Hkv, D))
    _check("v_cache", v_cache, k_cache.dtype, device, (S, Hkv, D))
    _check("page_table", page_table, torch.int32, device)
    if page_table.dim() != 2 or page_table.shape[0] != B:
        raise ValueError("page_table must be [B, P]")
    _check("seq_lens", seq_lens, torch.int32, device, (B,))
    if err_word is not None:
        _check_err_word(err_word, device)
    if lse is not None:
        _check("lse", lse, torch.float32, device, (B, Hq))
        if not lse.is_contiguous():
            raise ValueError("lse must be contiguous")
    if page_size < 1:
        raise ValueError("page_size must be positive")
    P = page_table.shape[1]
    if nsplit == 0:
        nsplit, need = qsa_paged_decode_plan(B, Hq, Hkv, D, P, page_size, _sm_count(device.index))
    else:
        nsplit, need = qsa_paged_decode_plan(B, Hq, Hkv, D, P, page_size, 0, nsplit)
    with _on(device, stream):
        if out is None:
            out = torch.empty(B, Hq, D, dtype=torch.bfloat16, device=device)
        else:
            _check("out", out, torch.bfloat16, device, (B, Hq, D))
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        elif workspace is not None:
            _check("workspace", workspace, torch.uint8, device)
        st = load_library().qsa_paged_decode(
            q.data_ptr(), q.stride(0), q.stride(1), k_cache.data_ptr(), k_cache.stride(0),
            k_cache.stride(1), v_cache.data_ptr(), v_cache.stride(0), v_cache.stride(1),
            page_table.data_ptr(), page_table.stride(0), seq_lens.data_ptr(), B, Hq, Hkv, D, P,
            S // page_size, page_size, 1.0 / (D ** 0.5) if scale is None else scale,
            1 if fp8 else 0, k_scale, v_scale, out.data_ptr(), out.stride(0), out.stride(1),
            _ptr(lse), nsplit, _ptr(workspace), workspace.numel() if workspace is not None else 0,
            _ptr(err_word), torch.cuda.current_stream(device).cuda_stream)
    if st != QSA_OK:
        _raise(st)
    return out
