"""Torch-facing calls of the operators around the selected-slot attention
(include/qsa_layer.h): the per-head norm and rotation that fills the cache, the index keys
of the cheap score, the selection of slots, and the attention of one new token over the
paged cache.  Like the rest of the package it turns tensors into pointers and computes
nothing; work is enqueued on ``stream`` (default: torch's current stream) and nothing is
synchronised.
"""
from __future__ import annotations

import ctypes
import importlib

import torch

from ._binding import QSAError, load_library, qsa_last_error_detail

_ext = None


def _load():
    """_layer_ext.so (built in-tree by build_lib.py): argument checks, allocation and the C call."""
    global _ext
    load_library()
    try:
        _ext = importlib.import_module("._layer_ext", __package__)
    except ImportError as e:
        raise RuntimeError("_layer_ext.so is missing or does not fit this torch: build it with "
                           "`python -m top_sparse_attention_index_b200.build_lib`") from e
    return _ext


def _call(name, stream, *args):
    ext = _ext or _load()
    if stream is None:
        r = getattr(ext, name)(*args)
    else:
        if args[0].is_cuda and stream.device != args[0].device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {args[0].device}")
        with torch.cuda.stream(stream):  # buffers allocated inside belong to the stream that uses them
            r = getattr(ext, name)(*args)
    if type(r) is int and r != 0:
        raise QSAError(r, qsa_last_error_detail())
    return r


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
    k_cache / v_cache [S, Hkv, D], bf16 or float8_e4m3fn (then multiplied by 1 / k_scale or
    1 / v_scale, a 32-bit number, and saturated).  Without k_cache the rotated keys come back as a new tensor.  q_out may
    be q.  Returns (q_out, rotated keys or None).
    """
    return _call("qk_norm_rope", stream, q, positions, inv_freq, k, v, q_weight, k_weight, eps, weight_offset,
                 sections, interleaved, rope_scale, q_out, k_cache, v_cache, slots, k_scale, v_scale, err_word)


def pack_index_keys(keys, blocks, codes, scales, block=4, err_word=None, stream=None):
    """int8 codes and scales of the cheap score's keys, one per named micro-block.

    keys bf16 [S, Di]: one index key per cache slot; blocks int32 [n]: physical micro-blocks
    (slot // block; -1 is skipped); codes int8 [S // block, Di] and scales float32
    [S // block] are written in place for the named blocks.  Returns (codes, scales).
    """
    _call("pack_index_keys", stream, keys, blocks, codes, scales, block, err_word)
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
    return _call("select_slots", stream, q, weight, codes, scales, page_table, seq_lens, top_blocks, page_size,
                 block, cu_q, sink_blocks, local_blocks, slot_idx, width, workspace, err_word)


def qsa_paged_decode_plan(B, Hq, Hkv, D, P, page_size, kv_fp8, num_sms, blocks_request=0):
    """(blocks, workspace_bytes) for this shape; raises QSAError for invalid shapes."""
    ws = ctypes.c_size_t(0)
    n = int(load_library().qsa_paged_decode_plan(B, Hq, Hkv, D, P, page_size, 1 if kv_fp8 else 0,
                                                 num_sms, blocks_request, ctypes.byref(ws)))
    if n < 0:
        raise QSAError(-n, qsa_last_error_detail())
    return n, int(ws.value)


def paged_decode(q, k_cache, v_cache, page_table, seq_lens, page_size, scale=None, k_scale=1.0,
                 v_scale=1.0, out=None, lse=None, blocks=0, workspace=None, err_word=None,
                 stream=None):
    """Attention of one new token per sequence over its whole paged cache.

    q [B, Hq, 256] bf16; k_cache / v_cache [S, Hkv, 256] bf16 or float8_e4m3fn (dequantised
    as code * k_scale, v_scale); page_table int32 [B, P]: token i of sequence b lies in slot
    page_table[b, i // page_size] * page_size + i % page_size; seq_lens int32 [B]; scale
    defaults to 1/16.  Returns out [B, Hq, 256] bf16 (zeros for an empty sequence); lse
    (float32 [B, Hq], optional) receives the base-2 log-sum-exp of the scaled scores.
    """
    return _call("paged_decode", stream, q, k_cache, v_cache, page_table, seq_lens, page_size, scale, k_scale,
                 v_scale, out, lse, blocks, workspace, err_word)
