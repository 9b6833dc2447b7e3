"""The layer operators where rounding, memory order or a failing wait decides the result:
calls that follow each other without a pause, scores a step apart, exact counts of slots."""
from __future__ import annotations

import math
import threading

import numpy as np
import pytest
import torch

import layer_reference as ref
import top_sparse_attention_index_b200 as qsa
from test_layer_gpu import (BF, F8, I32, check_select, close, decode_case, err_word, gen, keyed_case, normal,
                            rope_case, run_select, select_case)

pytestmark = pytest.mark.gpu


# ---- calls without a pause --------------------------------------------------------------------

def select_state(seed, lens, rows, Hi=4, Di=128, block=4, page=64):
    """Arguments of select_slots: sequences of `lens` tokens, each with its last rows[b] rows."""
    g = gen(seed)
    B, P = len(lens), -(-max(lens) // page)
    pool = B * P + 3
    S = pool * page
    codes = torch.zeros(S // block, Di, dtype=torch.int8, device="cuda")
    scales = torch.zeros(S // block, device="cuda")
    qsa.pack_index_keys(normal(g, S, Di), torch.arange(S // block, device="cuda", dtype=I32), codes, scales, block=block)
    cu = torch.tensor([sum(rows[:b]) for b in range(B + 1)], dtype=I32, device="cuda")
    Tq = sum(rows)
    return dict(q=normal(g, Tq, Hi, Di), weight=torch.randn(Tq, Hi, generator=g, device="cuda"), codes=codes,
                scales=scales, page_table=torch.randperm(pool, generator=g, device="cuda")[:B * P].to(I32).view(B, P),
                seq_lens=torch.tensor(lens, dtype=I32, device="cuda"), page_size=page, block=block, cu_q=cu)


LONG = ([65536], [7810])                                        # one long prefill
SHORT = ([8192, 8192], [8192, 8192])                            # rows of at most 2,048 blocks, a warp each
DECODE = ([65536 - 700 * b for b in range(64)], [1] * 64)       # a row per sequence


@pytest.mark.parametrize("lens,rows", [LONG, SHORT, DECODE], ids=["long", "short", "decode"])
def test_select_states_in_turn_over_one_workspace(lens, rows):
    """Calls on three inputs in turn, nothing between them, all in one workspace: each gives what
    a call of its own gives (scores of the call before, read in place of this one's, differ)."""
    top, turns = 512, 20
    states = [select_state(200 + i, [n - 64 * i for n in lens], rows) for i in range(3)]
    P = states[0]["page_table"].shape[1]
    need = qsa.qsa_select_slots_workspace_bytes(sum(rows), len(rows), P, 64, 4, 128, 4)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    want = []
    for s in states:
        want.append(qsa.select_slots(**s, top_blocks=top))
        torch.cuda.synchronize()
    outs = [[(torch.empty_like(i), torch.empty_like(w)) for i, w in want] for _ in range(turns)]
    torch.cuda.synchronize()
    for turn in outs:
        for s, (idx, width) in zip(states, turn):
            qsa.select_slots(**s, top_blocks=top, slot_idx=idx, width=width, workspace=work)
    torch.cuda.synchronize()
    for turn in outs:
        for (idx, width), (want_idx, want_width) in zip(turn, want):
            assert torch.equal(idx, want_idx) and torch.equal(width, want_width)


def test_index_keys_and_selection_in_turn():
    """Keys packed for the selection that follows at once, into the codes that the selection
    before has just read; the lengths and the page table change with them."""
    states = [select_state(210 + i, [9000 - 500 * i, 3000], [300, 1]) for i in range(3)]
    keys = [normal(gen(220 + i), states[0]["codes"].shape[0] * 4, 128) for i in range(3)]
    blocks = torch.arange(states[0]["codes"].shape[0], device="cuda", dtype=I32)
    shared = {k: states[0][k].clone() for k in ("codes", "scales", "page_table", "seq_lens")}

    def step(i, sync):
        for k in ("page_table", "seq_lens"):
            shared[k].copy_(states[i][k])
        qsa.pack_index_keys(keys[i], blocks, shared["codes"], shared["scales"])
        if sync:
            torch.cuda.synchronize()
        return qsa.select_slots(**{**states[i], **shared}, top_blocks=100)

    states = [dict(s, page_table=torch.nn.functional.pad(s["page_table"], (0, 141 - s["page_table"].shape[1])))
              for s in states]
    shared["page_table"] = torch.zeros_like(states[0]["page_table"])
    want = [step(i, True) for i in range(3)]
    torch.cuda.synchronize()
    got = [step(n % 3, False) for n in range(90)]
    torch.cuda.synchronize()
    for n, (idx, width) in enumerate(got):
        assert torch.equal(idx, want[n % 3][0]) and torch.equal(width, want[n % 3][1])


# ---- the score's roundings --------------------------------------------------------------------

def plain_select(s, top, rows_at_once=512):
    """select_slots of one sequence in elementary torch operations, every row: the products of
    codes exact (below 2^24), every other product and sum rounded to 32 bits, heads in order."""
    q, block, page = s["q"], s["block"], s["page_size"]
    Tq, Hi, _ = q.shape
    per, n = page // block, int(s["seq_lens"][0])

    def codes_of(x):
        step = x.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device="cuda")
        return torch.where(step > 0, torch.round(x / step), 0.0), step.squeeze(-1)

    code, step = codes_of(q.float())
    gain = s["weight"] * step
    where = (s["page_table"][0].long()[:, None] * per + torch.arange(per, device="cuda")).flatten()
    key, scale = s["codes"][where].double(), s["scales"][where]
    j = torch.arange(where.numel(), device="cuda")
    W = top * block + block - 1
    idx, width = torch.full((Tq, W), -1, dtype=I32, device="cuda"), torch.empty(Tq, dtype=I32, device="cuda")
    for t0 in range(0, Tq, rows_at_once):
        t = torch.arange(t0, min(Tq, t0 + rows_at_once), device="cuda")
        seen = (n - (Tq - 1 - t)).clamp(min=0)
        f = (seen // block)[:, None]
        dot = (code[t].double().flatten(0, 1) @ key.T).clamp(min=0).float().view(t.numel(), Hi, -1)
        total = gain[t, 0, None] * dot[:, 0]
        for h in range(1, Hi):
            total = total + gain[t, h, None] * dot[:, h]
        score = (total * scale).masked_fill(j >= f, float("-inf"))
        best = score.sort(dim=-1, descending=True, stable=True).indices[:, :top]
        best = torch.where(torch.arange(best.shape[1], device="cuda") < f, best, where.numel()).sort(-1).values
        taken = torch.minimum(f, torch.tensor(top, device="cuda"))
        slots = torch.cat([where, where.new_zeros(1)])[best][..., None] * block + torch.arange(block, device="cuda")
        idx[t, :slots.shape[1] * block] = slots.masked_fill((best == where.numel())[..., None], -1).flatten(1).to(I32)
        for e in range(block - 1):  # the incomplete block
            row = (e < seen - f[:, 0] * block).nonzero().flatten()
            idx[t[row], (taken[row, 0] * block + e)] = (where[f[row, 0]] * block + e).to(I32)
        width[t] = (taken[:, 0] * block + seen % block).to(I32)
    return idx, width


def test_select_every_row_of_a_long_prefill():
    """Of 7,810 rows over 16,384 blocks some have their border between scores a step apart."""
    for seed in range(230, 238):
        s = select_state(seed, *LONG)
        idx, width = qsa.select_slots(**s, top_blocks=512)
        want_idx, want_width = plain_select(s, 512)
        assert torch.equal(width, want_width)
        assert torch.equal(idx, want_idx), f"{int((idx != want_idx).any(1).sum())} rows differ"


@pytest.mark.parametrize("Hi", [1, 2, 3, 4, 7, 8, 16, 23, 32, 40, 64])
@pytest.mark.parametrize("Di", [64, 128])
def test_select_scores_a_step_apart(Hi, Di):
    """Blocks whose scores are 1 to within eight 32-bit steps: their order, and the choice, hang on
    every single rounding.  Many rows of a sequence and the same rows as sequences of their own."""
    n, rows = 700, 150
    s = select_state(240, [4 * n + 3], [rows], Hi, Di)
    s["q"] = s["q"][:1].expand(rows, Hi, Di).contiguous()
    s["weight"] = s["weight"][:1].abs().expand(rows, Hi).contiguous()  # (positive: no cancellation)
    where = (s["page_table"][0].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten()
    code, step = ref.codes_of(s["q"][0].float().cpu().numpy())
    gain = s["weight"][0].double() * torch.from_numpy(step).cuda().double()
    total = ((torch.from_numpy(code).cuda().double() @ s["codes"][where].double().T).clamp(min=0) * gain[:, None]).sum(0)
    wobble = 1 + torch.randint(0, 8, total.shape, generator=gen(241), device="cuda") * 2.0 ** -23
    s["scales"][where] = torch.where(total > 0, wobble / total, 1.0).float()
    top = 200
    want_idx, want_width = plain_select(s, top)
    idx, width = qsa.select_slots(**s, top_blocks=top)
    assert torch.equal(idx, want_idx) and torch.equal(width, want_width)
    alone = dict(s, cu_q=None, page_table=s["page_table"].expand(rows, -1).contiguous(),
                 seq_lens=4 * n + 3 - (rows - 1) + torch.arange(rows, device="cuda", dtype=I32))
    idx, width = qsa.select_slots(**alone, top_blocks=top)
    assert torch.equal(idx, want_idx) and torch.equal(width, want_width)


# ---- scores of no size ------------------------------------------------------------------------

def zeros_case(n, rows):
    """`rows` rows of one sequence of n blocks: scores of +0, of a negative product that underflows
    (-0), and a few below zero; all zeros are equal, so the lower blocks win."""
    c = keyed_case(torch.ones(n, device="cuda"), rows, 0)
    c["weight"].fill_(-1e-10)
    kind = torch.randint(0, 5, c["scales"].shape, generator=gen(250), device="cuda")
    c["scales"] = torch.tensor([0.0, 1e-40, 0.0, 1e-40, 1.0], device="cuda")[kind]
    return c


@pytest.mark.parametrize("rows,n", [(1, 700), (150, 700), (1300, 700), (1, 40000), (200, 40000), (1300, 40000)])
def test_select_zeros_of_both_signs_are_equal(rows, n):
    """In both forms of the score, and in the choice of short and long rows; of the long ones more
    blocks share the border than are collected."""
    c = zeros_case(n, rows)
    if n == 700 and rows == 1300:  # rows of at most 2,048 blocks, a warp each
        c["seq_lens"] += rows
        c["page_table"] = torch.cat([c["page_table"], c["page_table"][:, :1].expand(1, 21)], 1).contiguous()
    for top, sink, local in ((100, 0, 0), (500, 1, 7)):
        got, width = run_select(c, top, sink, local)
        for t in sorted({0, rows // 2, rows - 1}):
            want, want_width = ref.select(c["q"][t:t + 1], c["weight"][t:t + 1], c["codes"], c["scales"],
                                          c["page_table"], c["seq_lens"] - (rows - 1 - t), None, top,
                                          c["page_size"], 1, sink, local)
            assert torch.equal(got[t].cpu(), torch.from_numpy(want[0])) and int(width[t]) == int(want_width[0])


def test_select_scores_that_underflow():
    """Scores of both signs from 2^-130 down, subnormal ones and zeros among them."""
    for rows in (None, [140, 70]):
        c = select_case(251, [3000, 2500], rows, 4, 128, 4, 64)
        c["weight"] = (c["weight"] * 1e-10).contiguous()
        c["scales"] = torch.exp2(-100 - 30 * torch.rand(c["scales"].shape, generator=gen(252), device="cuda"))
        assert check_select(c, 100) == 0 and check_select(c, 500, 1, 3) == 0


def test_select_ignores_what_the_workspace_held():
    """The score's room full of NaNs of both signs, infinities and -0 before the call."""
    c = select_case(253, [3000, 2500], [140, 3], 4, 128, 4, 64)
    P = c["page_table"].shape[1]
    work = torch.empty(qsa.qsa_select_slots_workspace_bytes(143, 2, P, 64, 4, 128, 4), dtype=torch.uint8, device="cuda")
    want, want_width = run_select(c, 100)
    for bits in (0x7fffffff, -1, 0x7f800000, -2 ** 31):
        work[:work.numel() // 4 * 4].view(I32).fill_(bits)
        got, width = run_select(c, 100, workspace=work)
        assert torch.equal(got, want) and torch.equal(width, want_width)


@pytest.mark.parametrize("cu", [[0, 60, 20, 100], [0, 3, 1, 4], [0, 300] + [0, 300] * 6, [300, 0, 300]])
def test_select_offsets_that_decrease_are_reported(cu):
    """Sequences that share rows: an error bit, and nothing outside the pool."""
    B, Tq = len(cu) - 1, max(cu)
    c = select_case(254, [3000] * B, [-(-Tq // B)] * B, 4, 128, 4, 64)
    c["q"], c["weight"] = c["q"][:Tq], c["weight"][:Tq]
    c["cu_q"] = torch.tensor(cu, dtype=I32, device="cuda")
    err = err_word()
    idx, width = run_select(c, 100, err_word=err)
    assert int(err) == qsa.QSA_ERRBIT_WIDTH_RANGE
    in_use = width >= 0  # (a row of no sequence keeps -7)
    assert (idx[in_use] >= -1).all() and (idx < c["codes"].shape[0] * 4).all()
    assert (width[in_use] <= 403).all() and in_use.sum() > 0


# ---- waits that run out -----------------------------------------------------------------------

@pytest.mark.parametrize("rows", [[300, 140], [1500, 9]])
def test_select_waits_that_run_out(rows):
    """The tcgen05 score with a limit of its waits below the latency of what they wait for: the call
    ends, its rows are empty and the error word says so, and the next call is right."""
    c = select_case(260, [6000, 5000], rows, 4, 128, 4, 64)
    want, want_width = run_select(c, 100)
    torch.cuda.synchronize()
    lib = qsa.load_library()
    late = 0
    for ns in (0, 0, 100, 300, 1000, 3000, 10000, 30000):
        before = lib.qsa_probe_select_wait_ns(ns)
        try:
            err = err_word()
            got, width = run_select(c, 100, err_word=err)
            torch.cuda.synchronize()
        finally:
            lib.qsa_probe_select_wait_ns(before)
        assert before == 10 ** 9
        if int(err) == qsa.QSA_ERRBIT_TIMEOUT:
            late += 1
            assert (got == -1).all() and (width == 0).all()
        else:
            assert int(err) == 0 and torch.equal(got, want) and torch.equal(width, want_width)
        err = err_word()
        got, width = run_select(c, 100, err_word=err)
        assert int(err) == 0 and torch.equal(got, want) and torch.equal(width, want_width)
    assert late > 0


# ---- two host threads -------------------------------------------------------------------------

def select_call(c, top, stream):
    """A call of the C entry point with everything but its execution done beforehand, and its outputs."""
    lib = qsa.load_library()
    Tq, Hi, Di = c["q"].shape
    B, P = c["page_table"].shape
    block, page = c["block"], c["page_size"]
    W = top * block + block - 1
    idx = torch.full((Tq, W), -7, dtype=I32, device="cuda")
    width = torch.full((Tq,), -7, dtype=I32, device="cuda")
    need = qsa.qsa_select_slots_workspace_bytes(Tq, B, P, page, Hi, Di, block)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    cu = None if c["cu_q"] is None else c["cu_q"].data_ptr()
    args = (c["q"].data_ptr(), c["q"].stride(0), c["q"].stride(1), c["weight"].data_ptr(), c["weight"].stride(0),
            c["codes"].data_ptr(), c["codes"].stride(0), c["scales"].data_ptr(), c["page_table"].data_ptr(), P,
            c["seq_lens"].data_ptr(), cu, Tq, B, P, c["codes"].shape[0] * block // page, page, Hi, Di, block, top, 0, 0,
            idx.data_ptr(), W, width.data_ptr(), work.data_ptr(), need, None, stream.cuda_stream)
    return lambda: lib.qsa_select_slots(*args), idx, width, work


@pytest.mark.parametrize("rows", [None, [1300]])
def test_select_from_two_host_threads(rows):
    """A small and a large call again and again, each in its own thread and stream: no launch of
    one is refused for the shared memory that the other asks for."""
    lens = [9000] if rows is None else [1900]
    a = select_case(270, lens, rows, 64, 64, 1, 64)   # four groups of heads; thousands of blocks taken
    b = select_case(271, [300], None if rows is None else [1300], 10, 64, 1, 64)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    jobs = [select_call(a, 1800, streams[0]), select_call(b, 8, streams[1])]
    torch.cuda.synchronize()
    status = [set(), set()]

    def work(i):
        for _ in range(500):
            status[i].add(jobs[i][0]())

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert status == [{0}, {0}]
    for c, top, (_, idx, width, _) in ((a, 1800, jobs[0]), (b, 8, jobs[1])):
        want, want_width = ref.select(c["q"], c["weight"], c["codes"], c["scales"], c["page_table"], c["seq_lens"],
                                      c["cu_q"], top, 64, 1, 0, 0)
        assert torch.equal(idx.cpu(), torch.from_numpy(want)) and torch.equal(width.cpu(), torch.from_numpy(want_width))


# ---- decode: every slot counts once -----------------------------------------------------------

def share_borders(lens, fp8, groups):
    """Positions (per sequence) of the first and last tokens of every thread block's share."""
    unit = 64 if fp8 else 32  # slots that the work is shared out in
    units = [-(-n // unit) for n in lens]
    total = sum(units)
    groups = min(total, groups)
    marks = [{0, n - 1} if n else set() for n in lens]
    for c in range(1, groups):
        u = c * (total // groups) + min(c, total % groups)
        for b, n in enumerate(units):
            if u < n:
                marks[b] |= {max(u * unit - 1, 0), u * unit}
                break
            u -= n
    return marks


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens", [[100003], [30011, 12, 0, 8000, 4097, 1, 31, 33, 64, 65], [4096] * 40,
                                  [(37 * b) % 200 for b in range(700)]], ids=["one", "ragged", "equal", "many"])
@pytest.mark.parametrize("blocks", [0, 4, 28, 2000])
def test_decode_counts_every_slot_once(lens, blocks, fp8):
    """Scores of 0: every weight is 1, so the log-sum-exp is log2 of the length, and a value that
    only one slot holds comes out divided by the length.  The marked slots are the first and last
    ones of the thread blocks' shares, 256 per KV head.

    The log-sum-exp: two approximate logarithms (2^-22 of at most 17 each) and their roundings,
    exponentials of differences of the pieces' (2^-18): below 2^-17 + 2^-18; one slot of 100,003
    is 2^-16.1.  The values: approximations and 32-bit sums below 2^-16, bf16 2^-8: 2^-7 in all."""
    Hkv, page = 4, 64
    c = decode_case(280, lens, 2 * Hkv, Hkv, page, fp8)
    plan, _ = qsa.qsa_paged_decode_plan(len(lens), 2 * Hkv, Hkv, 256, c["page_table"].shape[1], page, fp8,
                                        torch.cuda.get_device_properties(0).multi_processor_count, blocks)
    marks = share_borders(lens, fp8, plan // Hkv)
    c["v_cache"] = torch.zeros_like(c["v_cache"].float())
    want = torch.zeros(len(lens), Hkv, 256, dtype=torch.float64, device="cuda")
    value = 256.0
    for b, n in enumerate(lens):
        at = sorted(marks[b])
        at = at[::-(-len(at) // (256 * Hkv))] if at else at
        if not at:
            continue
        slots = ref.slots_of(c["page_table"][b], n, page, 10 ** 9)[torch.tensor(at, device="cuda")]
        k = torch.arange(len(at), device="cuda")
        c["v_cache"][slots, k // 256, k % 256] = value
        want[b, k // 256, k % 256] = value * c.get("v_scale", 1.0) / n
    c["v_cache"] = c["v_cache"].to(F8 if fp8 else BF)
    lse = torch.full((len(lens), 2 * Hkv), 7.0, device="cuda")
    out = qsa.paged_decode(**c, scale=0.0, lse=lse, blocks=blocks)
    want = want.repeat_interleave(2, 1)
    close(out, want, 2.0 ** -7 * want)
    n = torch.tensor(lens, dtype=torch.float64, device="cuda")
    want_lse = torch.log2(n)[:, None].expand_as(lse)
    assert torch.equal(lse[n == 0], want_lse[n == 0].float())
    assert ((lse.double() - want_lse)[n > 0].abs() <= 2.0 ** -17 + 2.0 ** -18).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("log2", [22.5, 25.5])
def test_decode_of_dominant_tokens_keeps_the_rest(log2, fp8):
    """262,144 tokens in one thread block; the first token of each warp outweighs every other one
    by 2^22.5 or 2^25.5, and the output is what the others sum to (their values are 1, its is 0).

    Off by, of the output: a weight 2^-8 (bf16) or 2^-25 of the largest weight's 2^7, a 16-bit
    float's half step; the numerator's sum, 17 addends at a time cut at 2^-24 of it, over 2^13
    steps of half its size on average: 2^-8; the store 2^-8; the denominator, by what it may
    lose: addends below 2^-24 of a 32-bit sum, at most the others' share."""
    n = 262144
    c = decode_case(281, [n], 1, 1, 64, fp8, extra_pages=0)
    warps = 4 if fp8 else 2
    one, zero = torch.tensor([1.0, 0.0]).to(F8 if fp8 else BF)
    c["k_scale"] = c["v_scale"] = 1.0
    c["q"] = torch.ones_like(c["q"])
    for name, first, others in (("k_cache", one, zero), ("v_cache", zero, one)):
        x = c[name].view(torch.uint8)
        x[:] = others.view(1).view(torch.uint8).cuda().repeat(256)
        slots = ref.slots_of(c["page_table"][0], n, 64, 10 ** 9)[torch.arange(warps, device="cuda") * 16]
        x[slots] = first.view(1).view(torch.uint8).cuda().repeat(256)
    lse = torch.zeros(1, 1, device="cuda")
    out = qsa.paged_decode(**c, scale=log2 * math.log(2) / 256, lse=lse, blocks=1).double()
    rest = (n - warps) * 2.0 ** -log2
    want, share = rest / (warps + rest), rest / warps
    weight = 2.0 ** (log2 - 32) if fp8 else 2.0 ** -8
    assert ((out - want).abs() <= want * (weight + 2.0 ** -8 + 2.0 ** -8 + share)).all(), (out.min(), out.max(), want)
    # between the dominant tokens' alone and the whole sum's
    assert math.log2(warps) - 2.0 ** -17 <= float(lse) - log2 <= math.log2(warps + rest * (1 + weight)) + 2.0 ** -17


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 15, 16, 17, 33, 300, 5000])
@pytest.mark.parametrize("blocks", [0, 2, 50])
def test_decode_keeps_a_nan(n, blocks, fp8):
    """A NaN in the last key of one KV head, or in a query, comes out in every element of the heads
    that read it, whatever the length and the split; the others are untouched."""
    nan = torch.tensor([0x7f], dtype=torch.uint8, device="cuda") if fp8 else \
        torch.full((1,), float("nan"), dtype=BF, device="cuda").view(torch.uint8)
    for what in ("key", "query", "first query"):
        c = decode_case(282, [n, n + 3], 6, 2, 16, fp8)
        clean_lse = torch.zeros(2, 6, device="cuda")
        clean = qsa.paged_decode(**c, lse=clean_lse, blocks=blocks)
        hit = torch.zeros(2, 6, dtype=torch.bool, device="cuda")
        if what == "key":
            slot = ref.slots_of(c["page_table"][0], n, 16, 10 ** 9)[-1]
            c["k_cache"].view(torch.uint8)[slot, 1, :nan.numel()] = nan
            hit[0, 3:] = True
        else:
            c["q"] = c["q"].clone()
            c["q"][0, 0 if what == "first query" else 4, 77] = float("nan")
            hit[0, 0 if what == "first query" else 4] = True
        lse = torch.zeros(2, 6, device="cuda")
        out = qsa.paged_decode(**c, lse=lse, blocks=blocks)
        assert out[hit].isnan().all() and lse[hit].isnan().all()
        assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


# ---- index keys of hardly any size ------------------------------------------------------------

@pytest.mark.parametrize("block", [1, 3, 8, 9, 11, 15, 16])
def test_pack_index_keys_of_subnormal_means(block):
    """Means of 2^-133 and little more over the block: the scale keeps few bits, a quotient can be
    128 and more, and a code is at most 127 in magnitude, with its value's sign."""
    n = 64
    k = torch.arange(1, n + 1, device="cuda").double() * 2.0 ** -133  # exact bf16 subnormals (to 2^-126) and normals
    keys = torch.zeros(n, block, 64, dtype=BF, device="cuda")
    keys[:, 0, 0] = k.to(BF)
    keys[:, 0, 5] = -k.to(BF)
    keys[:, block - 1, 9] = (k / 2).to(BF)
    codes, scales = torch.zeros(n, 64, dtype=torch.int8, device="cuda"), torch.zeros(n, device="cuda")
    qsa.pack_index_keys(keys.view(n * block, 64), torch.arange(n, dtype=I32, device="cuda"), codes, scales, block=block)
    x = keys.float().cpu().numpy()
    mean = (x[:, 0] if block == 1 else x[:, 0] + x[:, block - 1]) / np.float32(block)
    scale = np.abs(mean).max(-1) / np.float32(127)
    want = np.clip(np.rint(mean / scale[:, None]), -127, 127)
    assert mean.dtype == scale.dtype == np.float32 and (scale > 0).all()
    assert torch.equal(scales.cpu(), torch.from_numpy(scale))
    assert torch.equal(codes.cpu(), torch.from_numpy(want.astype(np.int8)))
    assert (codes[:, 0] > 0).all() and (codes[:, 5] < 0).all()


# ---- a cache without a slot -------------------------------------------------------------------

@pytest.mark.parametrize("fp8", [False, True])
def test_norm_rope_into_an_empty_pool(fp8):
    """No token has a slot: queries are turned as ever, nothing is stored, a slot is reported."""
    c = rope_case(290, 5, 4, 2, 128, 64, 1)
    want, _ = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"])
    pool = torch.zeros(0, 2, 128, dtype=F8 if fp8 else BF, device="cuda")
    for slot, bits in ((-1, 0), (0, qsa.QSA_ERRBIT_SLOT_RANGE)):
        err = err_word()
        got, keys = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], k=c["k"], v=c["v"], k_cache=pool,
                                     v_cache=pool, slots=torch.full((5,), slot, dtype=I32, device="cuda"), err_word=err)
        assert torch.equal(got, want) and keys is None and int(err) == bits


# ---- different calls at once, and one workspace of several graphs -----------------------------

def test_different_calls_at_once():
    """Two streams, each with selections and decodes of its own in turn."""
    jobs = [(select_state(300 + i, [9000 - 64 * i, 3000], [300, 200 + i]), decode_case(310 + i, [9000, 40 + i], 16, 2, 64,
                                                                                     i % 2 == 1)) for i in range(4)]
    want = []
    for s, d in jobs:
        want.append((*qsa.select_slots(**s, top_blocks=100), qsa.paged_decode(**d)))
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for turn in range(12):
        for i, stream in enumerate(streams):
            n = 2 * i + turn % 2
            s, d = jobs[n]
            got.append((n, (*qsa.select_slots(**s, top_blocks=100, stream=stream), qsa.paged_decode(**d, stream=stream))))
    torch.cuda.synchronize()
    for n, outs in got:
        assert all(torch.equal(a, b) for a, b in zip(outs, want[n]))


def test_graphs_that_share_a_workspace():
    """Captured calls of different inputs over one workspace, replayed in turn without a pause."""
    states = [select_state(320 + i, [9000 - 64 * i, 3000], [300, 200]) for i in range(3)]
    caches = [decode_case(330 + i, [9000 - i, 40], 16, 2, 64) for i in range(3)]
    sizes = [qsa.qsa_select_slots_workspace_bytes(500, 2, 141, 64, 4, 128, 4),
             qsa.qsa_paged_decode_plan(2, 16, 2, 256, 142, 64, False, 148, 0)[1]]
    work = torch.empty(max(sizes) * 2, dtype=torch.uint8, device="cuda")
    want, outs, graphs = [], [], []
    for s, d in zip(states, caches):
        want.append((*qsa.select_slots(**s, top_blocks=100), qsa.paged_decode(**d)))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((*qsa.select_slots(**s, top_blocks=100, workspace=work), qsa.paged_decode(**d, workspace=work)))
        graphs.append(graph)
    for _ in range(8):
        for out in outs:
            for x in out:
                x.fill_(-5)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out, exp in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, exp))
