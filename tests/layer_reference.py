"""Plain 64-bit references of the layer operators (include/qsa_layer.h), with the error
bounds that their roundings allow.

A rounding is off by at most half a step: relative 2^-8 for bf16, 2^-11 for fp16, 2^-24 for
fp32, 2^-4 for E4M3 (below its smallest normal value, 2^-10 absolute).
"""
from __future__ import annotations

import math

import numpy as np
import torch


# ---- norm and rotation ----------------------------------------------------------------------

def norm_rope(x, weight, offset, eps, positions, inv_freq, sections, interleaved, rope_scale):
    """(y, slack): the normed and rotated rows of x [T, H, D] in float64 and the absolute error
    that 32-bit arithmetic may leave in them before the store's rounding.

    The slack counts, relative to |u| + |v| of a pair: the mean of squares (8 terms per lane and
    at most 5 shuffled sums: 13 roundings, halved by the root), root, reciprocal, the weight's
    sum and three products (6), the angle in fp32 turns (2 pi 2^-25 < 2^-22), sine and cosine
    (2 ulp, 2^-23 each), their scale and the rotation's three operations (4): below 25 * 2^-24
    + 2^-21 < 2^-18."""
    T, H, D = x.shape
    y = x.double()
    if weight is not None:
        y = y / (y.pow(2).mean(-1, keepdim=True) + eps).sqrt() * (weight.double() + offset)
    half = inv_freq.numel()
    if half == 0:
        return y, y.abs() * 2.0 ** -18
    pos = positions.double().reshape(-1, T)
    axis = [0] * half if sections is None else [a for a, n in enumerate(sections) for _ in range(n)]
    angle = pos[axis].T * inv_freq.double()                       # [T, half]
    c, s = rope_scale * angle.cos()[:, None], rope_scale * angle.sin()[:, None]
    first = torch.arange(half, device=x.device) * (2 if interleaved else 1)
    second = first + (1 if interleaved else half)
    u, v = y[..., first], y[..., second]
    out, slack = y.clone(), y.abs()
    out[..., first], out[..., second] = u * c - v * s, v * c + u * s
    slack[..., first] = slack[..., second] = (u.abs() + v.abs()) * max(1.0, abs(rope_scale))
    return out, slack * 2.0 ** -18


def bf16_tolerance(ref, slack):
    return (ref.abs() + slack) * 2.0 ** -8 + slack


def e4m3_tolerance(ref, slack):
    """Of codes of `ref` (already divided by the scale, and saturated)."""
    return torch.maximum((ref.abs() + slack) * 2.0 ** -4, torch.full_like(ref, 2.0 ** -10)) + slack


# ---- the cheap score ------------------------------------------------------------------------

def pack(keys, block):
    """(codes, scales) of bf16 keys [n * block, Di] as float32 numpy arithmetic, step by step."""
    x = keys.float().cpu().numpy().reshape(-1, block, keys.shape[-1])
    with np.errstate(all="ignore"):
        total = x[:, 0].copy()
        for e in range(1, block):
            total = total + x[:, e]
        mean = (total / np.float32(block)).astype(np.float32)
        return codes_of(mean)


def codes_of(x):
    with np.errstate(all="ignore"):
        scale = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
        scale = np.where(np.isfinite(scale), scale, np.float32(np.nan)).astype(np.float32)
        q = np.rint((x / scale[..., None]).astype(np.float32))
        q = np.where((scale > 0)[..., None], q, 0)
    return q.astype(np.int8), scale


def select(q, weight, codes, scales, table, lens, cu, top, page, block, sink, local):
    """(slot_idx, width) row by row; rows of no sequence are -7.  Integer dots, then float32
    products and sums in head order."""
    q = q.float().cpu().numpy()
    weight, codes, scales = weight.cpu().numpy(), codes.cpu().numpy().astype(np.int64), scales.cpu().numpy()
    table, lens = table.cpu().numpy(), lens.cpu().numpy()
    Tq, Hi, _ = q.shape
    B, P = table.shape
    cu = np.arange(B + 1) if cu is None else cu.cpu().numpy()
    per, pages = page // block, codes.shape[0] // (page // block)
    if pages == 0:  # an empty pool: every page lies outside it
        codes, scales = np.zeros((1, codes.shape[1]), np.int64), np.zeros(1, np.float32)
    W = top * block + block - 1
    out, width = np.full((Tq, W), -7, np.int32), np.full(Tq, -7, np.int32)
    qc, qs = codes_of(q)
    for b in range(B):
        n = min(max(int(lens[b]), 0), P * page)
        for t in range(cu[b], cu[b + 1]):
            seen = max(n - (cu[b + 1] - 1 - t), 0)
            f = seen // block
            j = np.arange(f)
            pg = table[b, j // per].astype(np.int64) if f else np.zeros(0, np.int64)
            ok = (pg >= 0) & (pg < pages)
            phys = np.where(ok, pg * per + j % per, 0)
            dots = np.maximum(qc[t].astype(np.int64) @ codes[phys].T, 0).astype(np.float32)
            with np.errstate(all="ignore"):
                gain = (weight[t] * qs[t]).astype(np.float32)
                s = (gain[0] * dots[0]).astype(np.float32)
                for h in range(1, Hi):
                    s = (s + (gain[h] * dots[h]).astype(np.float32)).astype(np.float32)
                s = (s * scales[phys]).astype(np.float64)
            s[np.isnan(s) | ~ok] = -np.inf
            rank = np.where((j < sink) | (j >= f - local), 0, 1)
            order = np.lexsort((j, -s, rank))[:top]
            row = []
            for k in sorted(order):
                base = int(pg[k]) * page + int(k % per) * block
                row += [base + e if ok[k] else -1 for e in range(block)]
            tail = seen - f * block
            if tail:
                p = int(table[b, f // per])
                good = 0 <= p < pages
                row += [p * page + (f % per) * block + e if good else -1 for e in range(tail)]
            width[t] = len(row)
            out[t] = row + [-1] * (W - len(row))
    return out, width


# ---- attention over the paged cache ---------------------------------------------------------

def slots_of(table_row, n, page, pages):
    """Physical slots of a sequence's n tokens, without those of pages outside the pool."""
    i = torch.arange(n, device=table_row.device)
    pg = table_row.long()[i // page]
    ok = (pg >= 0) & (pg < pages)
    return (pg * page + i % page)[ok]


def paged_decode(q, k_cache, v_cache, table, lens, page, scale, k_scale=1.0, v_scale=1.0):
    """(out, tolerance, lse) in float64.

    The tolerance: the weights p are rounded to 16 bits (relative d = 2^-8 for bf16, 2^-11 for
    fp16, there also 2^-25 absolute below 2^-14 against a largest weight of at least 1) in
    numerator and denominator alike, which moves the mean by at most d / (1 - d) sum w |v - out|;
    the scores' 32-bit sums of 256 products add 2^-16 scale sum |q k| to d; sums over the slots
    in 32 bits, the exponential, the joins and the scales stay below 2^-16 sum w |v|; the store rounds to
    bf16, 2^-8."""
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    G = Hq // Hkv
    fp8 = k_cache.dtype == torch.float8_e4m3fn
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    tol = torch.zeros_like(out)
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device=q.device)
    pages = k_cache.shape[0] // page
    for b in range(B):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        slots = slots_of(table[b], n, page, pages)
        if slots.numel() == 0:
            continue
        for j in range(Hkv):
            k = k_cache[:, j].view(torch.uint8 if fp8 else torch.bfloat16)[slots]
            v = v_cache[:, j].view(torch.uint8 if fp8 else torch.bfloat16)[slots]
            if fp8:
                k, v = k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
            k, v = k.double() * k_scale, v.double() * v_scale
            h = slice(j * G, (j + 1) * G)
            qs = q[b, h].double()
            s = qs @ k.T * scale
            w = torch.softmax(s, -1)
            o = w @ v
            spread = torch.stack([(w[g][:, None] * (v - o[g]).abs()).sum(0) for g in range(G)])
            d = (2.0 ** -11 if fp8 else 2.0 ** -8) + 2.0 ** -16 * abs(scale) * (qs.abs() @ k.abs().T).amax()
            small = 2.0 ** -25 * v.abs().sum(0) if fp8 else 0.0
            err = d / (1 - d) * spread + 2.0 ** -16 * (w @ v.abs()) + small
            out[b, h], tol[b, h] = o, err + 2.0 ** -8 * (o.abs() + err)
            lse[b, h] = torch.logsumexp(s, -1) / math.log(2.0)
    return out, tol, lse
