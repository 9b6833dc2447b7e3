"""The operators around the selected-slot attention in a serving layer, and the calls that
measure them.

Four operators: the per-head norm and rotation that fills the cache (``rotate``), the
packing of index keys (``index``), the selection of slots by a cheap score (``select``) and
the attention of one new token over the paged cache (``decode``).  ``run`` computes them in
elementary torch operations, or through the package's entry points where ``own`` is true.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

D = 256  # head dimension of the attention


# ---- the cases --------------------------------------------------------------------------

def _rotate(**kw):
    case = dict(op="rotate", tokens=16, heads=16, kv_heads=2, dim=D, rot=64, pairs="halves",
                axes=1, cache="bf16")
    return {**case, **kw}


def _index(**kw):
    case = dict(op="index", blocks=64, block=4, dim=128, holes=False)
    return {**case, **kw}


def _select(**kw):
    case = dict(op="select", seqs=1, rows=1, length=65536, ragged=False, heads=4, dim=128, block=4,
                page=64, top=512, sink=0, local=0)
    return {**case, **kw}


def _decode(**kw):
    case = dict(op="decode", seqs=1, length=1500, ragged=False, heads=16, kv_heads=2, page=64,
                cache="bf16")
    return {**case, **kw}


def listed():
    return [
        # one decode step of a batch: a row per sequence, latency counts
        _rotate(name="rotate_decode_16"),
        # two requests of 8,192 positions prefilled together
        _rotate(name="rotate_prefill_16384", tokens=16384, heads=24),
        # a ragged prefill with image tokens: time, height and width positions, fp8 cache
        _rotate(name="rotate_axes_e4m3_5003", tokens=5003, heads=12, kv_heads=1, axes=3, cache="e4m3"),
        # one decode step: some sequences complete a micro-block, the others do not
        _index(name="index_decode_64", holes=True),
        # the micro-blocks of a 262,144-slot cache after a long prefill
        _index(name="index_prefill_65536", blocks=65536),
        # one decode step of a batch over ragged long caches
        _select(name="select_decode_64", seqs=64, ragged=True),
        # one sequence at the largest extent
        _select(name="select_decode_1", length=262144 - 3, sink=1, local=32),
        # two requests of 8,192 positions prefilled together, most recent blocks kept
        _select(name="select_two_requests", seqs=2, rows=8192, length=8192, local=32),
        # the last 7,810 rows of a 65,536-token prompt
        _select(name="select_long_prefill", rows=7810),
        # one sequence, a short cache: latency counts
        _decode(name="decode_1"),
        # a batch of ragged sequences
        _decode(name="decode_batch_64", seqs=64, length=8192, ragged=True, heads=24),
        # a few sequences at the largest extent, fp8 cache
        _decode(name="decode_long_e4m3", seqs=4, length=262144, cache="e4m3"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


SHAPES = ((16, 2), (24, 2), (12, 1), (6, 1), (3, 1), (8, 8), (16, 1))  # query and KV heads


def draw(rng):
    op = rng.choice(("rotate", "index", "select", "select", "decode", "decode"))
    if op == "rotate":
        heads, kv_heads = rng.choice(SHAPES)
        return _rotate(tokens=_log_int(rng, 1, 12000), heads=heads, kv_heads=kv_heads,
                       dim=(dim := rng.choice((D, D, 128))), rot=rng.choice((32, 64, 128, dim)), pairs=rng.choice(("halves", "neighbours")),
                       axes=rng.choice((1, 1, 3)), cache=rng.choice(("bf16", "e4m3")))
    if op == "index":
        return _index(blocks=_log_int(rng, 1, 50000), block=rng.choice((1, 2, 4, 4, 8, 16)),
                      dim=rng.choice((64, 128)), holes=rng.random() < 0.5)
    if op == "select":
        block = rng.choice((1, 2, 4, 4, 4, 8))
        page = block * rng.choice((1, 3, 4, 16, 16, 64))
        common = dict(block=block, page=page, dim=rng.choice((64, 128, 128)),
                      heads=rng.choice((1, 2, 4, 4, 8, 16)), top=_log_int(rng, 8, 2048 // block),
                      sink=rng.choice((0, 0, 1)), local=rng.choice((0, 0, 7)))
        if rng.random() < 0.5:  # decode steps
            return _select(seqs=_log_int(rng, 1, 64), length=_log_int(rng, 1, 65536),
                           ragged=rng.random() < 0.7, **common)
        rows = _log_int(rng, 2, 2000)
        return _select(seqs=rng.choice((1, 1, 2, 3)), rows=rows,
                       length=rows + _log_int(rng, 1, 20000), **common)
    heads, kv_heads = rng.choice(SHAPES)
    seqs = _log_int(rng, 1, 100)
    return _decode(seqs=seqs, length=_log_int(rng, 1, 262144 // seqs), ragged=rng.random() < 0.7,
                   heads=heads, kv_heads=kv_heads, page=rng.choice((1, 16, 24, 64, 100, 256)),
                   cache=rng.choice(("bf16", "e4m3")))


# ---- inputs -----------------------------------------------------------------------------

K_SCALE, V_SCALE = 0.0135, 0.0125  # per-tensor scales that put N(0, 1) values near the format's maximum


def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


def _lengths(case, gen):
    """Tokens of each sequence: all the same, or between an eighth of it and all of it."""
    B, n = case["seqs"], case["length"]
    if not case["ragged"]:
        return torch.full((B,), n, dtype=torch.int32, device="cuda")
    lens = torch.randint(max(1, n // 8), n + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    lens[0] = n
    return lens


def _pages(case, gen):
    """A page table in which every sequence owns pages in random places of the pool."""
    per = -(-case["length"] // case["page"])
    pool = case["seqs"] * per + 3
    order = torch.randperm(pool, generator=gen, device="cuda")[:case["seqs"] * per]
    return order.to(torch.int32).reshape(case["seqs"], per), pool


def _codes(x):
    """int8 codes and the scale of each last-dimension vector of fp32 values."""
    top = x.abs().amax(-1, keepdim=True)
    s = top / torch.full_like(top, 127.0)  # by a number it would be a product with the reciprocal
    c = torch.where(s > 0, torch.round(x / s), torch.zeros_like(x))
    return c, s.squeeze(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op == "rotate":
        T, H, J, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        qkv = _normal(gen, T, (H + 2 * J) * d)  # one row of the projection per token
        s["q"] = qkv[:, :H * d].view(T, H, d)
        s["k"] = qkv[:, H * d:(H + J) * d].view(T, J, d)
        s["v"] = qkv[:, (H + J) * d:].view(T, J, d)
        s["q_weight"] = 1 + 0.1 * _normal(gen, d)
        s["k_weight"] = 1 + 0.1 * _normal(gen, d)
        pos = torch.randint(0, 262144 - T, (case["axes"], 1), generator=gen, device="cuda")
        steps = torch.arange(T, device="cuda")
        # the axes of image tokens advance at different rates
        s["pos"] = torch.stack([pos[a] + steps // (24 ** a) for a in range(case["axes"])]).to(torch.int32)
        if case["axes"] == 1:
            s["pos"] = s["pos"][0]
        half = case["rot"] // 2
        s["inv_freq"] = (1e7 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)).float()
        # a third each to height and width, the rest to time
        s["sections"] = (half - 2 * (half // 3), half // 3, half // 3) if case["axes"] == 3 else None
        slots = torch.randperm(T + 37, generator=gen, device="cuda")[:T].to(torch.int32)
        slots[T // 2 + 1::97] = -1  # rows of padding: nothing is stored
        s["slots"] = slots
        s["k_cache"], s["v_cache"] = _normal(gen, T + 37, J, d), _normal(gen, T + 37, J, d)
        if case["cache"] == "e4m3":
            s["k_cache"] = s["k_cache"].to(torch.float8_e4m3fn)
            s["v_cache"] = s["v_cache"].to(torch.float8_e4m3fn)
    elif op == "index":
        n, block = case["blocks"], case["block"]
        total = n + 11
        s["keys"] = _normal(gen, total * block, case["dim"])
        ids = torch.randperm(total, generator=gen, device="cuda")[:n].to(torch.int32)
        if case["holes"]:
            ids[1::4] = -1
        s["ids"] = ids
        s["codes"] = torch.zeros(total, case["dim"], dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(total, device="cuda")
    elif op == "select":
        B, L, block = case["seqs"], case["rows"], case["block"]
        s["table"], pool = _pages(case, gen)
        s["lens"] = _lengths(case, gen)
        s["cu"] = torch.arange(B + 1, device="cuda", dtype=torch.int32) * L
        s["q"] = _normal(gen, B * L, case["heads"], case["dim"])
        s["weight"] = torch.randn(B * L, case["heads"], generator=gen, device="cuda")
        keys = _normal(gen, pool * case["page"] // block, block, case["dim"]).float()
        codes, s["scales"] = _codes(keys.mean(1))
        s["codes"] = codes.to(torch.int8)
    else:
        B, J = case["seqs"], case["kv_heads"]
        s["table"], pool = _pages(case, gen)
        s["lens"] = _lengths(case, gen)
        s["q"] = _normal(gen, B, case["heads"], D)
        for name, scale in (("k", K_SCALE), ("v", V_SCALE)):
            cache = _normal(gen, pool * case["page"], J, D)
            if case["cache"] == "e4m3":
                cache = (cache.float() / scale).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[name + "_cache"] = cache
    return s


# ---- one pass ---------------------------------------------------------------------------

def run(state):
    if own:
        import top_sparse_attention_index_b200 as qsa
        return _own(qsa, state)
    return {"rotate": _plain_rotate, "index": _plain_index, "select": _plain_select,
            "decode": _plain_decode}[state["op"]](state)


def _own(qsa, s):
    op = s["op"]
    if op == "rotate":
        q, _ = qsa.qk_norm_rope(s["q"], s["pos"], s["inv_freq"], k=s["k"], v=s["v"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"], sections=s["sections"],
                                interleaved=s["pairs"] == "neighbours", k_cache=s["k_cache"],
                                v_cache=s["v_cache"], slots=s["slots"], k_scale=K_SCALE, v_scale=V_SCALE)
        return q, s["k_cache"], s["v_cache"]
    if op == "index":
        qsa.pack_index_keys(s["keys"], s["ids"], s["codes"], s["scales"], block=s["block"])
        return s["codes"], s["scales"]
    if op == "select":
        return qsa.select_slots(s["q"], s["weight"], s["codes"], s["scales"], s["table"], s["lens"],
                                top_blocks=s["top"], page_size=s["page"], block=s["block"],
                                cu_q=s["cu"], sink_blocks=s["sink"], local_blocks=s["local"])
    return qsa.paged_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                            page_size=s["page"], k_scale=K_SCALE, v_scale=V_SCALE)


def _axis_of_pair(s):
    """The axis whose position turns each pair: contiguous sections."""
    half = s["rot"] // 2
    if s["sections"] is None:
        return torch.zeros(half, dtype=torch.long, device="cuda")
    return torch.repeat_interleave(torch.arange(3, device="cuda"),
                                   torch.tensor(s["sections"], device="cuda"), output_size=half)


def _turn(x, s, cos, sin):
    """The rotation of the first `rot` dimensions; cos and sin are [tokens, 1, rot / 2]."""
    rot = s["rot"]
    if s["pairs"] == "halves":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    else:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    return torch.cat((turned, x[..., rot:]), -1)


def _plain_rotate(s):
    pos = s["pos"].reshape(s["axes"], -1).double()
    angle = pos[_axis_of_pair(s)].T * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def normed(x, w):
        x = x.float()
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()

    q = _turn(normed(s["q"], s["q_weight"]), s, cos, sin).to(torch.bfloat16)
    k = _turn(normed(s["k"], s["k_weight"]), s, cos, sin)
    v = s["v"].float()
    if s["cache"] == "e4m3":
        k, v = (k / K_SCALE).clamp(-448, 448), (v / V_SCALE).clamp(-448, 448)
    keep = s["slots"] >= 0
    at = s["slots"][keep].long()
    for cache, x in ((s["k_cache"], k), (s["v_cache"], v)):
        x = x[keep].to(cache.dtype)
        if cache.dtype == torch.float8_e4m3fn:  # stored as bytes
            cache.view(torch.uint8)[at] = x.view(torch.uint8)
        else:
            cache[at] = x
    return q, s["k_cache"], s["v_cache"]


def _plain_index(s):
    keep = s["ids"] >= 0
    at = s["ids"][keep].long()
    x = s["keys"].view(-1, s["block"], s["dim"])[at].float()
    total = functools.reduce(torch.add, x.unbind(1))  # in slot order
    codes, scales = _codes(total / s["block"])
    s["codes"][at] = codes.to(torch.int8)
    s["scales"][at] = scales
    return s["codes"], s["scales"]


def _visible(s):
    """[seqs, rows] tokens that each row sees, its own included."""
    L = s["rows"]
    return s["lens"].long()[:, None] - (L - 1) + torch.arange(L, device="cuda")[None]


def _physical(s, per):
    """[seqs, n] physical number of every logical unit, `per` units to a page."""
    return (s["table"].long()[:, :, None] * per + torch.arange(per, device="cuda")).flatten(1)


def _chosen(s, score):
    """Slots of the blocks that `score` [seqs, rows, blocks] picks, and their number."""
    B, L, n = score.shape
    block, top = s["block"], s["top"]
    seen = _visible(s)
    full = (seen // block)[..., None]
    j = torch.arange(n, device="cuda")
    score = torch.where(score.isnan(), -math.inf, score)
    kept = (j < s["sink"]) | (j >= full - s["local"])
    score = torch.where(kept, math.inf, score)
    # a stable sort keeps the lower index first; invisible blocks come after every visible one
    order = score.masked_fill(j >= full, -math.inf).sort(dim=-1, descending=True, stable=True).indices
    order = order[..., :top]
    # visible blocks of the lowest score precede invisible ones: their indices are lower
    taken = torch.arange(order.shape[-1], device="cuda") < full
    blocks = torch.where(taken, order, n).sort(dim=-1).values
    where = torch.cat((_physical(s, s["page"] // block), torch.zeros_like(s["table"][:, :1]).long()), 1)
    W = top * block + block - 1
    out = torch.full((B, L, W), -1, dtype=torch.int32, device="cuda")
    slots = where.gather(1, blocks.flatten(1)).view(B, L, -1, 1) * block + torch.arange(block, device="cuda")
    slots = torch.where((blocks < n)[..., None], slots, -1).flatten(2)
    out[..., :slots.shape[-1]] = slots.to(torch.int32)
    count = torch.minimum(full, torch.tensor(top, device="cuda")).squeeze(-1) * block
    tail = torch.arange(block - 1, device="cuda")
    position = full * block + tail
    place = where.gather(1, (position // block).clamp(max=n).flatten(1)).view(B, L, -1) * block + tail
    inside = position < seen[..., None]
    at = (count[..., None] + tail).clamp(max=W - 1)
    old = out.gather(2, at)
    out.scatter_(2, at, torch.where(inside, place.to(torch.int32), old))
    return out.flatten(0, 1), (count + seen % block).to(torch.int32).flatten()


def _plain_select(s):
    B, L, H, d = s["seqs"], s["rows"], s["heads"], s["dim"]
    codes, step = _codes(s["q"].float())
    gain = (s["weight"] * step).view(B, L, H)
    where = _physical(s, s["page"] // s["block"])
    keys = s["codes"][where].float()  # [seqs, blocks, dim]
    # sums of at most 128 products of whole numbers up to 127: exact in 32 bits
    dots = (codes.view(B, L * H, d) @ keys.transpose(1, 2)).view(B, L, H, -1).relu_()
    # each product and each sum of the score rounded to 32 bits, heads in order
    total = functools.reduce(torch.add, (gain[:, :, h, None] * dots[:, :, h] for h in range(H)))
    return _chosen(s, total * s["scales"][where][:, None])


def _plain_decode(s):
    B, H, J = s["seqs"], s["heads"], s["kv_heads"]
    where = _physical(s, s["page"])
    q = s["q"].float().view(B, J, H // J, D)
    fp8 = s["cache"] == "e4m3"

    def rows(cache):
        cache = cache.view(torch.uint8)[where].view(cache.dtype) if fp8 else cache[where]
        return cache.float().transpose(1, 2)  # [seqs, KV heads, slots, D]

    score = q @ rows(s["k_cache"]).transpose(2, 3) * (D ** -0.5 * (K_SCALE if fp8 else 1.0))
    past = torch.arange(where.shape[1], device="cuda") >= s["lens"][:, None]
    score = score.masked_fill(past[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    out = p @ rows(s["v_cache"]) / p.sum(-1, keepdim=True) * (V_SCALE if fp8 else 1.0)
    return out.reshape(B, H, D).to(torch.bfloat16)


# ---- what a pass cannot do without ------------------------------------------------------

def _mean_length(case):
    return case["length"] * (9 / 16 if case["ragged"] and case["seqs"] > 1 else 1)


def work(case):
    op = case["op"]
    if op == "rotate":
        rows, kv = case["tokens"] * case["dim"], 2 * case["kv_heads"]
        e = 1 if case["cache"] == "e4m3" else 2
        return {"bytes": rows * (4 * case["heads"] + kv * (2 + e)),
                "flops": rows * 7 * (case["heads"] + case["kv_heads"])}
    if op == "index":
        n = case["blocks"] * (0.75 if case["holes"] else 1)
        elements = n * case["block"] * case["dim"]
        return {"bytes": 2 * elements + n * (case["dim"] + 8), "flops": elements + 3 * n * case["dim"]}
    if op == "select":
        B, L = case["seqs"], case["rows"]
        n = _mean_length(case) / case["block"]  # blocks of a sequence
        pairs = B * L * max(0.0, n - (L - 1) / (2 * case["block"]))
        width = case["top"] * case["block"] + case["block"] - 1
        return {"bytes": B * n * (case["dim"] + 4) + B * L * (case["heads"] * (2 * case["dim"] + 4) + 4 * width + 4),
                "flops": pairs * case["heads"] * 2 * case["dim"]}
    slots = case["seqs"] * _mean_length(case)
    e = 1 if case["cache"] == "e4m3" else 2
    return {"bytes": 2 * slots * case["kv_heads"] * D * e + 4 * case["seqs"] * case["heads"] * D,
            "flops": 4 * slots * case["heads"] * D}


# ---- the definitions in 64 bits ---------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotate":
        return _exact_rotate(s)
    if op == "index":
        return _exact_index(s)
    if op == "select":
        # the score's own roundings make the choice: _exact_select repeats them one by one
        return _exact_select(s) if s["seqs"] * s["rows"] * s["length"] <= 1 << 26 else None
    return _exact_decode(s)


def _exact_rotate(s):
    """Each pair as a complex number times exp(i angle)."""
    rot, half = s["rot"], s["rot"] // 2
    pos = s["pos"].reshape(s["axes"], -1).double()
    axis = [0] * half if s["sections"] is None else sum(([a] * n for a, n in enumerate(s["sections"])), [])
    angle = pos[axis].T * s["inv_freq"].double()
    unit = torch.polar(torch.ones_like(angle), angle)[:, None]
    first = torch.arange(half, device="cuda") * (1 if s["pairs"] == "halves" else 2)
    second = first + (half if s["pairs"] == "halves" else 1)

    def turned(x, w):
        x = x.double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / s["dim"] + 1e-6).sqrt() * w.double()
        z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * unit
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    got = [turned(s["q"], s["q_weight"])]
    fp8 = s["cache"] == "e4m3"
    rows = torch.nonzero(s["slots"] >= 0).flatten()
    for cache, x, scale in ((s["k_cache"], turned(s["k"], s["k_weight"]), K_SCALE),
                            (s["v_cache"], s["v"].double(), V_SCALE)):
        x = (x / scale).clamp(-448, 448) if fp8 else x
        got.append(cache.double().index_copy_(0, s["slots"][rows].long(), x[rows]))
    return tuple(got)


def _exact_index(s):
    ids = s["ids"][s["ids"] >= 0].long()
    mean = s["keys"].double().view(-1, s["block"], s["dim"])[ids].mean(1)
    scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
    scales[ids] = mean.abs().amax(1) / 127
    # the code is a rounding of the value over the stored 32-bit scale: no 64-bit value of its own
    return None, scales


def _exact_select(s):
    """Row by row of sequences, sums in integers, each later step rounded once to 32 bits."""
    B, L, H, block = s["seqs"], s["rows"], s["heads"], s["block"]

    def f32(x):
        return x.float().double()

    q = s["q"].double()
    step = f32(q.abs().amax(-1) / 127)
    code = torch.where(step[..., None] > 0, f32(q / step[..., None]).round(), 0.0)
    gain = f32(s["weight"].double() * step)
    scores = []
    for b in range(B):
        pages = s["table"][b].long()
        unit = s["page"] // block
        phys = (pages.repeat_interleave(unit) * unit + torch.arange(unit, device="cuda").repeat(len(pages)))
        dot = torch.einsum("lhd,nd->lhn", code[b * L:(b + 1) * L], s["codes"][phys].double()).clamp(min=0)
        total = torch.zeros(L, len(phys), dtype=torch.float64, device="cuda")
        for h in range(H):
            total = f32(total + f32(gain[b * L:(b + 1) * L, h, None] * dot[:, h]))
        scores.append(f32(total * s["scales"][phys].double()))
    return _chosen(s, torch.stack(scores))


def _exact_decode(s):
    """Sequence by sequence over the slots that its pages name."""
    fp8 = s["cache"] == "e4m3"
    G = s["heads"] // s["kv_heads"]
    got = torch.zeros(s["seqs"], s["heads"], D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(s["lens"].tolist()):
        i = torch.arange(n, device="cuda")
        slots = s["table"][b].long()[i // s["page"]] * s["page"] + i % s["page"]
        for j in range(s["kv_heads"]):
            k = s["k_cache"][:, j].view(torch.uint8 if fp8 else torch.bfloat16)[slots]
            v = s["v_cache"][:, j].view(torch.uint8 if fp8 else torch.bfloat16)[slots]
            if fp8:
                k, v = k.view(torch.float8_e4m3fn).double() * K_SCALE, v.view(torch.float8_e4m3fn).double() * V_SCALE
            heads = slice(j * G, (j + 1) * G)
            w = torch.softmax(s["q"][b, heads].double() @ k.double().T / 16, -1)
            got[b, heads] = w @ v.double()
    return got
