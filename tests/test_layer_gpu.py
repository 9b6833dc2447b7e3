"""The layer operators (include/qsa_layer.h) on the GPU against the 64-bit references of
layer_reference.py, at the sizes and masks where they can go wrong, and a run of them
together: rows into the cache, index keys, selection, attention over the selection, and the
attention of the next token over the whole cache."""
from __future__ import annotations

import pytest
import torch

import layer_reference as ref
import top_sparse_attention_index_b200 as qsa

pytestmark = pytest.mark.gpu

BF, I32, F8 = torch.bfloat16, torch.int32, torch.float8_e4m3fn
SLOT_RANGE, WIDTH_RANGE, Q_RANGE = qsa.QSA_ERRBIT_SLOT_RANGE, qsa.QSA_ERRBIT_WIDTH_RANGE, qsa.QSA_ERRBIT_Q_RANGE


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").to(BF)


def err_word():
    return torch.zeros(1, dtype=I32, device="cuda")


def close(got, want, tol):
    got = got.double()
    bad = ~((got - want).abs() <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} of {bad.numel()}; first at {i}: got {got[i].item()}, "
                             f"want {want[i].item()} within {tol[i].item()}")


# ---- norm and rotation ----------------------------------------------------------------------

def rope_case(seed, T, Hq, Hkv, D, rot, axes):
    g = gen(seed)
    qkv = normal(g, T, (Hq + 2 * Hkv) * D + 8)[:, 8:]  # rows of a wider projection
    half = rot // 2
    c = dict(q=qkv[:, :Hq * D].view(T, Hq, D), k=qkv[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D),
             v=qkv[:, (Hq + Hkv) * D:].view(T, Hkv, D), q_weight=1 + 0.1 * normal(g, D),
             k_weight=1 + 0.1 * normal(g, D))
    c["positions"] = torch.randint(0, 262144, (T,) if axes == 1 else (axes, T), generator=g, device="cuda", dtype=I32)
    c["inv_freq"] = (1e7 ** (-torch.arange(half, device="cuda").double() / max(half, 1))).float()
    c["sections"] = None if axes == 1 else [half - (axes - 1) * (half // axes)] + [half // axes] * (axes - 1)
    return c


def rope_want(c, name, offset=0.0, eps=1e-6, interleaved=False, rope_scale=1.0):
    return ref.norm_rope(c[name], c[name + "_weight"], offset, eps, c["positions"], c["inv_freq"], c["sections"],
                         interleaved, rope_scale)


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,axes,inter,fp8", [
    (1, 16, 2, 256, 64, 1, False, False), (17, 24, 2, 256, 256, 1, False, False), (33, 12, 1, 256, 64, 3, False, True),
    (5, 3, 1, 256, 128, 1, True, False), (40, 8, 8, 128, 128, 1, True, True), (9, 6, 1, 128, 32, 2, False, False),
    (70, 5, 3, 64, 64, 4, False, False), (11, 7, 2, 64, 16, 1, True, True), (3, 64, 8, 256, 0, 1, False, False),
    (2, 300, 1, 128, 96, 3, True, False), (1000, 16, 2, 256, 64, 1, False, True),
])
def test_norm_rope_into_the_cache(T, Hq, Hkv, D, rot, axes, inter, fp8):
    c = rope_case(1, T, Hq, Hkv, D, rot, axes)
    S = T + 9
    slots = torch.randperm(S, generator=gen(2), device="cuda")[:T].to(I32)
    slots[T // 2::7] = -1
    dt = F8 if fp8 else BF
    kv = normal(gen(3), S, 2, Hkv, D).to(dt)  # K and V rows of one packed cache
    before = kv.clone()
    ks, vs = 0.0135, 0.0125
    err = err_word()
    q, k_out = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], k=c["k"], v=c["v"], q_weight=c["q_weight"],
                                k_weight=c["k_weight"], sections=c["sections"], interleaved=inter, weight_offset=0.5,
                                rope_scale=1.25, k_cache=kv[:, 0], v_cache=kv[:, 1], slots=slots, k_scale=ks, v_scale=vs,
                                err_word=err)
    assert k_out is None and int(err) == 0
    want, slack = rope_want(c, "q", 0.5, interleaved=inter, rope_scale=1.25)
    close(q, want, ref.bf16_tolerance(want, slack))
    keep = slots >= 0
    at = slots[keep].long()
    want, slack = (x[keep] for x in rope_want(c, "k", 0.5, interleaved=inter, rope_scale=1.25))
    v = c["v"][keep].double()
    got = kv.view(torch.uint8)[at].view(dt)
    if fp8:
        # the quotient is one more 32-bit rounding, and so is the scale as a 32-bit argument
        want, slack, v = (want / ks).clamp(-448, 448), slack / ks + (want / ks).abs() * 2.0 ** -22, v / vs
        close(got[:, 0], want, ref.e4m3_tolerance(want, slack))
        v = v.clamp(-448, 448)
        close(got[:, 1], v, ref.e4m3_tolerance(v, v.abs() * 2.0 ** -22))
    else:
        close(got[:, 0], want, ref.bf16_tolerance(want, slack))
        assert torch.equal(got[:, 1], c["v"][keep])
    rest = torch.ones(S, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert torch.equal(kv.view(torch.uint8)[rest], before.view(torch.uint8)[rest])


def test_norm_rope_without_cache_weights_or_slots():
    c = rope_case(4, 37, 6, 2, 128, 64, 1)
    c["q_weight"] = c["k_weight"] = None
    q, k = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], k=c["k"])
    for name, got in (("q", q), ("k", k)):
        want, slack = rope_want(c, name)
        close(got, want, ref.bf16_tolerance(want, slack))
    # without slots row t goes to row t; the rows behind it stay
    cache = normal(gen(5), 40, 2, 128)
    before = cache.clone()
    qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], k=c["k"], k_cache=cache)
    assert torch.equal(cache[:37], k) and torch.equal(cache[37:], before[37:])
    only_q, none = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"])
    assert none is None and torch.equal(only_q, q)


def test_norm_rope_in_place():
    c = rope_case(6, 50, 16, 2, 256, 64, 1)
    args = dict(q_weight=c["q_weight"], k_weight=c["k_weight"])
    q, k = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], k=c["k"], **args)
    got, _ = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], k=c["k"], q_out=c["q"], k_cache=c["k"], **args)
    assert got is c["q"] and torch.equal(c["q"], q) and torch.equal(c["k"], k)


def test_norm_rope_far_and_negative_positions():
    c = rope_case(7, 8, 4, 1, 256, 64, 1)
    c["positions"] = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, 10 ** 9 + 7, 262143], dtype=I32,
                                  device="cuda")
    q, _ = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], q_weight=c["q_weight"])
    want, slack = rope_want(c, "q")
    close(q, want, ref.bf16_tolerance(want, slack))


def test_norm_rope_bad_slots_store_nothing():
    c = rope_case(8, 6, 4, 2, 256, 64, 1)
    kc, vc = normal(gen(9), 16, 2, 256), normal(gen(10), 16, 2, 256)
    kb, vb = kc.clone(), vc.clone()
    for bad in (16, -2, 2 ** 31 - 1, -2 ** 31):
        err = err_word()
        slots = torch.full((6,), -1, dtype=I32, device="cuda")
        slots[3] = bad
        qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], k=c["k"], v=c["v"], k_cache=kc, v_cache=vc, slots=slots,
                         err_word=err)
        assert int(err) == SLOT_RANGE
        assert torch.equal(kc, kb) and torch.equal(vc, vb)


def test_norm_rope_zero_rows_and_saturation():
    c = rope_case(11, 4, 2, 1, 64, 32, 1)
    c["q"][1] = 0
    c["v"][2] = 3.0e4
    kc, vc = torch.zeros(4, 1, 64, device="cuda").to(F8), torch.zeros(4, 1, 64, device="cuda").to(F8)
    q, _ = qsa.qk_norm_rope(c["q"], c["positions"], c["inv_freq"], k=c["k"], v=c["v"], q_weight=c["q_weight"],
                            k_cache=kc, v_cache=vc)
    assert (q[1] == 0).all() and (vc[2].float() == 448).all()
    empty, _ = qsa.qk_norm_rope(c["q"][:0], c["positions"][:0], c["inv_freq"])
    assert empty.shape == (0, 2, 64)


# ---- index keys -----------------------------------------------------------------------------

@pytest.mark.parametrize("block,Di,n", [(1, 128, 5), (2, 64, 33), (3, 128, 100), (4, 128, 64), (4, 64, 1), (7, 128, 3),
                                        (16, 64, 200), (13, 128, 4097)])
def test_pack_index_keys(block, Di, n):
    g = gen(20)
    total = n + 5
    keys = normal(g, total * block + block - 1, Di + 8)[:, :Di]  # strided rows, an incomplete block at the end
    keys[:block] = 0
    ids = torch.randperm(total, generator=g, device="cuda")[:n].to(I32)
    ids[n // 3::5] = -1
    codes = torch.full((total, Di + 16), 77, dtype=torch.int8, device="cuda")[:, :Di]
    scales = torch.full((total,), -3.0, device="cuda")
    err = err_word()
    qsa.pack_index_keys(keys, ids, codes, scales, block=block, err_word=err)
    assert int(err) == 0
    want_c, want_s = ref.pack(keys[:total * block], block)
    named = torch.zeros(total, dtype=torch.bool)
    named[ids[ids >= 0].long().cpu()] = True
    assert torch.equal(codes.cpu()[named], torch.from_numpy(want_c)[named])
    assert torch.equal(scales.cpu()[named], torch.from_numpy(want_s)[named])
    assert (codes.cpu()[~named] == 77).all() and (scales.cpu()[~named] == -3.0).all()


def test_pack_index_keys_out_of_range_and_not_finite():
    keys = normal(gen(21), 42, 64)  # ten blocks of four, two rows beyond
    keys[4, 3], keys[9, 60], keys[13] = float("nan"), float("inf"), 1e-39
    codes, scales = torch.zeros(10, 64, dtype=torch.int8, device="cuda"), torch.zeros(10, device="cuda")
    err = err_word()
    ids = torch.tensor([1, 2, 3, 10, -2, 2 ** 31 - 1], dtype=I32, device="cuda")
    qsa.pack_index_keys(keys, ids, codes, scales, err_word=err)
    assert int(err) == SLOT_RANGE
    assert scales[1:3].isnan().all() and (codes[1:3] == 0).all()
    want_c, want_s = ref.pack(keys[12:16], 4)
    assert torch.equal(codes[3].cpu(), torch.from_numpy(want_c)[0]) and float(scales[3]) == float(want_s[0])
    assert (scales[[0, 4, 9]] == 0).all()


# ---- selection ------------------------------------------------------------------------------

def select_case(seed, lens, rows, Hi, Di, block, page, extra_pages=1, gap=0):
    """Sequences of the given lengths and row counts (None: one row each, no cu_q), `gap` rows of
    no sequence before and after."""
    g = gen(seed)
    B = len(lens)
    P = max(-(-n // page) for n in lens) + extra_pages
    pool = B * P + 2
    c = dict(block=block, page_size=page)
    c["page_table"] = torch.randperm(pool, generator=g, device="cuda")[:B * P].to(I32).view(B, P)
    c["seq_lens"] = torch.tensor(lens, dtype=I32, device="cuda")
    if rows is None:
        Tq, c["cu_q"] = B, None
    else:
        cu = [gap]
        for n in rows:
            cu.append(cu[-1] + n)
        Tq, c["cu_q"] = cu[-1] + gap, torch.tensor(cu, dtype=I32, device="cuda")
    c["q"] = normal(g, Tq, Hi + 1, Di)[:, :Hi]
    c["weight"] = torch.randn(Tq, Hi + 3, generator=g, device="cuda")[:, :Hi]
    codes, scales = ref.pack(normal(g, pool * page, Di), block)
    c["codes"], c["scales"] = torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda()
    return c


def run_select(c, top, sink=0, local=0, **kw):
    Tq = c["q"].shape[0]
    W = top * c["block"] + c["block"] - 1
    idx = torch.full((Tq, W + 5), -7, dtype=I32, device="cuda")
    width = torch.full((Tq,), -7, dtype=I32, device="cuda")
    qsa.select_slots(c["q"], c["weight"], c["codes"], c["scales"], c["page_table"], c["seq_lens"], top, c["page_size"],
                     block=c["block"], cu_q=c["cu_q"], sink_blocks=sink, local_blocks=local, slot_idx=idx[:, :W],
                     width=width, **kw)
    assert (idx[:, W:] == -7).all()
    return idx[:, :W], width


def check_select(c, top, sink=0, local=0):
    err = err_word()
    idx, width = run_select(c, top, sink, local, err_word=err)
    want_idx, want_width = ref.select(c["q"], c["weight"], c["codes"], c["scales"], c["page_table"], c["seq_lens"],
                                      c["cu_q"], top, c["page_size"], c["block"], sink, local)
    assert torch.equal(width.cpu(), torch.from_numpy(want_width))
    assert torch.equal(idx.cpu(), torch.from_numpy(want_idx))
    return int(err)


@pytest.mark.parametrize("Hi", [1, 2, 3, 4, 5, 8, 9, 16, 17, 33, 64])
@pytest.mark.parametrize("Di", [64, 128])
def test_select_heads(Hi, Di):
    """Every head count of a tile, one row per sequence and rows of a prefill."""
    assert check_select(select_case(30, [900, 5, 2001], None, Hi, Di, 4, 64), 40) == 0
    assert check_select(select_case(31, [900, 71, 2001], [130, 70, 3], Hi, Di, 4, 64), 40) == 0


@pytest.mark.parametrize("block,page", [(1, 1), (1, 64), (2, 6), (3, 48), (4, 4), (4, 100), (8, 64), (16, 256)])
def test_select_blocks_and_pages(block, page):
    c = select_case(32, [block * 150 + block - 1, block * 37, 3 * block], [21, 40, 1], 4, 128, block, page, gap=3)
    for top, sink, local in ((1, 0, 0), (24, 0, 0), (24, 1, 7), (30, 30, 0), (30, 0, 30)):
        check_select(c, top, sink, local)


@pytest.mark.parametrize("lens", [[0], [1], [3], [4], [5], [0, 0, 1, 4, 700], [163], [164], [165]])
def test_select_short_sequences(lens):
    """No token, no complete block, as many blocks as are taken (40) and one more."""
    assert check_select(select_case(33, lens, None, 4, 128, 4, 16), 40) == 0
    # more rows than tokens: the first rows see nothing
    assert check_select(select_case(34, lens, [n % 13 + 3 for n in lens], 4, 128, 4, 16, gap=2), 40) == 0


def test_select_rows_of_no_sequence_and_empty_sequences():
    c = select_case(35, [500, 300, 420, 10], [9, 0, 5, 0], 4, 128, 4, 64, gap=4)
    assert check_select(c, 16) == 0


def test_select_ties_go_to_the_lower_block():
    for codes in (0, 3):
        c = select_case(36, [4003, 2900], [10, 1], 4, 128, 4, 64)
        c["codes"].fill_(codes)
        c["scales"].fill_(0.5)
        check_select(c, 100)
    # a handful of different scores only
    c = select_case(37, [9001], [3], 2, 64, 1, 64)
    c["codes"].zero_()
    c["codes"][:, 0] = torch.randint(0, 3, (c["codes"].shape[0],), generator=gen(38), device="cuda", dtype=torch.int8)
    check_select(c, 1000, 1, 7)


def test_select_values_that_are_not_finite():
    c = select_case(39, [3000, 2500], [20, 1], 4, 128, 4, 64)
    n = c["scales"].numel()
    c["scales"][torch.randperm(n, generator=gen(40), device="cuda")[:n // 2]] = float("nan")
    c["scales"][7::31] = float("inf")
    c["weight"][3, 1] = float("-inf")
    c["weight"][4, 0] = float("nan")
    c["q"][5, 2, 7] = float("nan")
    c["q"][6, 1, 9] = float("inf")
    c["q"][7] = 0
    check_select(c, 300, 1, 7)
    check_select(c, 600)


def test_select_pages_outside_the_pool():
    c = select_case(41, [2000, 900], [40, 1], 4, 128, 4, 64)
    c["page_table"][0, 3], c["page_table"][0, 31], c["page_table"][1, 0] = -1, 10 ** 9, -2 ** 31
    assert check_select(c, 64) == SLOT_RANGE
    assert check_select(c, 490, 1, 0) == SLOT_RANGE  # more than the good blocks: the bad ones come out as -1


def test_select_lengths_and_offsets_outside_their_range():
    c = select_case(42, [500, 600], None, 4, 128, 4, 64)
    c["seq_lens"][0], c["seq_lens"][1] = -5, 2 ** 31 - 1
    assert check_select(c, 16) == WIDTH_RANGE
    c = select_case(43, [500, 600], [30, 20], 4, 128, 4, 64)
    good, _ = run_select(c, 16)
    c["cu_q"][0], c["cu_q"][2] = -3, 1000
    err = err_word()
    got, _ = run_select(c, 16, err_word=err)
    assert int(err) == WIDTH_RANGE
    assert torch.equal(got[:30], good[:30])  # the first sequence's last row is the same


def test_select_many_rows_in_chunks():
    """More rows than a chunk of scores holds, short sequences in a wide page table."""
    c = select_case(44, [1500, 700], [900, 120], 1, 64, 4, 64, extra_pages=9000)
    assert c["page_table"].shape[1] * 16 * 1020 * 4 > 512 << 20
    check_select(c, 32)


def test_select_long_row_takes_the_largest_budget():
    check_select(select_case(45, [70003], None, 2, 64, 1, 64), 8192, 1, 100)
    check_select(select_case(46, [262143], None, 1, 64, 4, 64), 2048)


def test_select_is_the_same_however_the_rows_are_batched():
    c = select_case(47, [3000, 2000], [70, 33], 4, 128, 4, 64)
    whole, width = run_select(c, 64)
    last = dict(c, q=c["q"][[69, 102]], weight=c["weight"][[69, 102]], cu_q=None)
    idx, w = run_select(last, 64)
    assert torch.equal(idx, whole[[69, 102]]) and torch.equal(w, width[[69, 102]])


# ---- decode ---------------------------------------------------------------------------------

def decode_case(seed, lens, Hq, Hkv, page, fp8=False, extra_pages=1, packed=False):
    g = gen(seed)
    B = len(lens)
    P = max(-(-max(n, 0) // page) for n in lens) + extra_pages
    pool = B * P + 2
    c = dict(page_size=page)
    c["page_table"] = torch.randperm(pool, generator=g, device="cuda")[:B * P].to(I32).view(B, P)
    c["seq_lens"] = torch.tensor(lens, dtype=I32, device="cuda")
    c["q"] = normal(g, B, 2, Hq, 256)[:, 1]
    kv = normal(g, pool * page, 2, Hkv, 256)
    if fp8:
        kv = (kv.float() / 0.013).clamp(-448, 448).to(F8)
        c["k_scale"], c["v_scale"] = 0.013, 0.0125
    if packed:
        c["k_cache"], c["v_cache"] = kv[:, 0], kv[:, 1]
    else:
        c["k_cache"], c["v_cache"] = (kv.view(torch.uint8)[:, i].contiguous().view(kv.dtype) for i in (0, 1))
    return c


def check_decode(c, **kw):
    B, Hq, _ = c["q"].shape
    err = err_word()
    lse = torch.full((B, Hq), 7.0, device="cuda")
    out = qsa.paged_decode(**c, lse=lse, err_word=err, **kw)
    scale = kw.get("scale", 1 / 16)
    want, tol, want_lse = ref.paged_decode(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["seq_lens"],
                                           c["page_size"], scale, c.get("k_scale", 1.0), c.get("v_scale", 1.0))
    close(out, want, tol)
    empty = torch.isinf(want_lse)
    assert torch.equal(empty, lse == float("-inf")) and (out[empty] == 0).all()
    # the rounded weights (2^-8) and 32-bit sums: 2^-7 in the natural logarithm
    assert ((lse - want_lse)[~empty].abs() <= 2.0 ** -6 + 2.0 ** -20 * want_lse[~empty].abs()).all()
    return int(err), out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 1), (6, 1), (8, 8), (12, 1), (16, 2), (24, 2), (16, 1), (45, 5)])
def test_decode_heads(Hq, Hkv, fp8):
    assert check_decode(decode_case(50, [333, 1, 0, 64, 65], Hq, Hkv, 16, fp8, packed=True))[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [1, 3, 16, 24, 100, 256])
@pytest.mark.parametrize("blocks", [0, 1, 3, 50])
def test_decode_pages_and_splits(page, blocks, fp8):
    check_decode(decode_case(51, [999, 15, 17, 128, 0, 500], 12, 2, page, fp8), blocks=blocks)


@pytest.mark.parametrize("n", [0, 1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 129])
def test_decode_short(n):
    check_decode(decode_case(52, [n], 16, 2, 64))
    check_decode(decode_case(53, [n], 16, 2, 64, True))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_long_and_ragged(fp8):
    check_decode(decode_case(54, [30011, 12, 8000, 4097], 24, 2, 64, fp8))
    check_decode(decode_case(55, [100003], 8, 1, 64, fp8))


def test_decode_short_sequences_in_a_wide_page_table():
    check_decode(decode_case(56, [70, 1000], 16, 2, 64, extra_pages=2000))


def test_decode_many_sequences():
    lens = torch.randint(0, 200, (700,), generator=torch.Generator().manual_seed(57)).tolist()
    check_decode(decode_case(57, lens, 3, 1, 16))


def test_decode_large_scores():
    """One slot outweighs all others by far; scores beyond 1,000."""
    c = decode_case(58, [300, 64], 16, 2, 16)
    c["q"].mul_(8)
    c["k_cache"].mul_(8)
    check_decode(c, scale=0.5)
    check_decode(c, scale=-0.5)
    check_decode(c, scale=0.0)


def test_decode_pages_outside_the_pool_are_masked():
    for fp8 in (False, True):
        c = decode_case(59, [300, 200, 90], 16, 2, 16, fp8)
        c["page_table"][0, 2], c["page_table"][0, 18], c["page_table"][1, :] = -1, 10 ** 9, -2 ** 31
        err, out = check_decode(c)
        assert err == SLOT_RANGE and (out[1] == 0).all()
        check_decode(c, blocks=5)


def test_decode_ignores_rows_behind_the_end():
    """NaN and infinity in slots that no length reaches, in pages that are half used."""
    for fp8 in (False, True):
        c = decode_case(60, [301, 77, 5], 16, 2, 64, fp8)
        keep = torch.zeros(c["k_cache"].shape[0], dtype=torch.bool, device="cuda")
        for b, n in enumerate([301, 77, 5]):
            keep[ref.slots_of(c["page_table"][b], n, 64, 10 ** 6)] = True
        for name in ("k_cache", "v_cache"):
            x = c[name].view(torch.uint8)
            x[~keep] = 0x7f if fp8 else 0xff  # NaN
        check_decode(c)


def test_decode_lengths_outside_their_range():
    c = decode_case(61, [100, 128], 8, 1, 16, extra_pages=0)
    c["seq_lens"][0], c["seq_lens"][1] = -1, 2 ** 31 - 1
    assert check_decode(c)[0] == WIDTH_RANGE


def test_decode_query_beyond_16_bit_floats_is_reported():
    c = decode_case(62, [100], 8, 1, 16, True)
    c["q"][0, 3, 5] = 65536.0
    err = err_word()
    qsa.paged_decode(**c, err_word=err)
    assert int(err) == Q_RANGE


def test_decode_is_bitwise_repeatable():
    c = decode_case(63, [9001, 300], 24, 2, 64)
    a, b = qsa.paged_decode(**c), qsa.paged_decode(**c)
    assert torch.equal(a, b)


def test_decode_offsets_beyond_32_bits():
    """Rows whose element offset passes 2^32."""
    page, Hkv = 64, 8
    pages = (2 ** 32 + 2 ** 20) // (page * Hkv * 256)
    k = torch.empty(pages * page, Hkv, 256, dtype=BF, device="cuda")
    table = torch.tensor([[pages - 1, 0, pages - 2]], dtype=I32, device="cuda")
    used = (table[0].long()[:, None] * page + torch.arange(page, device="cuda")).flatten()
    k[used] = normal(gen(64), used.numel(), Hkv, 256)
    c = dict(q=normal(gen(65), 1, 16, 256), k_cache=k, v_cache=k, page_table=table,
             seq_lens=torch.tensor([130], dtype=I32, device="cuda"), page_size=page)
    assert check_decode(c)[0] == 0


# ---- together -------------------------------------------------------------------------------

class Layer:
    """One layer's buffers: paged K / V cache, index keys and their codes."""

    def __init__(self, seed, lens, rows, Hq, Hkv, fp8):
        g = gen(seed)
        self.page, self.block, self.top, self.fp8 = 16, 4, 12, fp8
        self.lens, self.rows = lens, rows
        B, P = len(lens), max(lens) // 16 + 2
        pool = B * P + 1
        S = pool * 16
        self.table = torch.randperm(pool, generator=g, device="cuda")[:B * P].to(I32).view(B, P)
        self.seq_lens = torch.tensor(lens, dtype=I32, device="cuda")
        self.cu = torch.tensor([sum(rows[:i]) for i in range(B + 1)], dtype=I32, device="cuda")
        T = sum(rows)
        pos = torch.cat([torch.arange(n - r, n, device="cuda") for n, r in zip(lens, rows)])
        seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(rows, device="cuda"))
        self.pos = pos.to(I32)
        self.slots = (self.table[seq, pos // 16].long() * 16 + pos % 16).to(I32)
        done = (pos % 4 == 3)
        self.blocks = torch.where(done, self.slots // 4, -1).to(I32)
        self.freq = (1e4 ** (-torch.arange(32, device="cuda").double() / 32)).float()
        self.qkv = normal(g, T, Hq + 2 * Hkv, 256)
        self.q, self.k, self.v = self.qkv.split([Hq, Hkv, Hkv], 1)
        self.iq, self.iw = normal(g, T, 4, 128), torch.randn(T, 4, generator=g, device="cuda")
        self.wq, self.wk = 1 + 0.1 * normal(g, 256), 1 + 0.1 * normal(g, 256)
        dt = F8 if fp8 else BF
        self.scales = dict(k_scale=0.02, v_scale=0.0125) if fp8 else {}
        old = normal(g, S, 2, Hkv, 256).float() / (0.0125 if fp8 else 1.0)
        self.kc, self.vc = (old[:, i].clamp(-448, 448).to(dt) for i in (0, 1))
        self.ik = normal(g, S, 128)
        self.codes = torch.zeros(S // 4, 128, dtype=torch.int8, device="cuda")
        self.code_scales = torch.zeros(S // 4, device="cuda")
        qsa.pack_index_keys(self.ik, torch.arange(S // 4, dtype=I32, device="cuda"), self.codes, self.code_scales)
        self.err = err_word()

    def step(self):
        q, _ = qsa.qk_norm_rope(self.q, self.pos, self.freq, k=self.k, v=self.v, q_weight=self.wq, k_weight=self.wk,
                                k_cache=self.kc, v_cache=self.vc, slots=self.slots, err_word=self.err, **self.scales)
        qsa.pack_index_keys(self.ik, self.blocks, self.codes, self.code_scales, err_word=self.err)
        idx, width = qsa.select_slots(self.iq, self.iw, self.codes, self.code_scales, self.table, self.seq_lens,
                                      self.top, self.page, cu_q=self.cu, sink_blocks=1, local_blocks=2,
                                      err_word=self.err)
        sparse = qsa.sparse_prefill(q, self.kc, self.vc, idx, width, **self.scales)
        last = (self.cu[1:] - 1).long()
        dense = qsa.paged_decode(q[last], self.kc, self.vc, self.table, self.seq_lens, self.page, err_word=self.err,
                                 **self.scales)
        return q, idx, width, sparse, dense

    def check(self, got):
        q, idx, width, sparse, dense = got
        assert int(self.err) == 0
        want, slack = ref.norm_rope(self.q, self.wq, 0.0, 1e-6, self.pos, self.freq, None, False, 1.0)
        close(q, want, ref.bf16_tolerance(want, slack))
        want, slack = ref.norm_rope(self.k, self.wk, 0.0, 1e-6, self.pos, self.freq, None, False, 1.0)
        rows = self.kc.view(torch.uint8)[self.slots.long()].view(self.kc.dtype)
        if self.fp8:
            want, slack = (want / 0.02).clamp(-448, 448), slack / 0.02 + (want / 0.02).abs() * 2.0 ** -22
            close(rows, want, ref.e4m3_tolerance(want, slack))
        else:
            close(rows, want, ref.bf16_tolerance(want, slack))
        want_idx, want_width = ref.select(self.iq, self.iw, self.codes, self.code_scales, self.table, self.seq_lens,
                                          self.cu, self.top, self.page, 4, 1, 2)
        assert torch.equal(idx.cpu(), torch.from_numpy(want_idx))
        assert torch.equal(width.cpu(), torch.from_numpy(want_width))
        # a row's selection is a sequence of one-slot pages
        scale = (1 / 16, self.scales.get("k_scale", 1.0), self.scales.get("v_scale", 1.0))
        want, tol, _ = ref.paged_decode(q, self.kc, self.vc, idx, width, 1, *scale)
        close(sparse, want, tol)
        last = (self.cu[1:] - 1).long()
        want, tol, _ = ref.paged_decode(q[last], self.kc, self.vc, self.table, self.seq_lens, 16, *scale)
        close(dense, want, tol)


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_prefill_then_decode(fp8):
    layer = Layer(70, [203, 90, 17], [60, 1, 17], 24, 2, fp8)
    layer.check(layer.step())
    step = Layer(71, [300, 1, 6, 64], [1, 1, 1, 1], 16, 2, fp8)
    step.check(step.step())


def test_layer_step_in_two_graphs():
    """Two captured steps replayed in turn on new inputs, with eager calls between."""
    layers = [Layer(72, [203, 90], [1, 1], 16, 2, False), Layer(73, [500, 33, 8], [1, 1, 1], 16, 2, True)]
    graphs, outs = [], []
    for layer in layers:
        layer.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(layer.step())
        graphs.append(graph)
    for turn in range(2):
        for layer in layers:
            g = gen(80 + turn)
            layer.qkv.copy_(normal(g, *layer.qkv.shape))
            layer.iq.copy_(normal(g, *layer.iq.shape))
        for graph in graphs:
            graph.replay()
        for layer, out in zip(layers, outs):
            layer.check(out)
            layer.check(layer.step())


def test_calls_on_another_stream():
    """Each call on a stream of its own gives bitwise what the current stream gives."""
    layer = Layer(74, [203, 90, 17], [60, 1, 17], 16, 2, False)
    want = layer.step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    last = (layer.cu[1:] - 1).long()
    torch.cuda.synchronize()
    q, _ = qsa.qk_norm_rope(layer.q, layer.pos, layer.freq, k=layer.k, v=layer.v, q_weight=layer.wq, k_weight=layer.wk,
                            k_cache=layer.kc, v_cache=layer.vc, slots=layer.slots, stream=s)
    idx, width = qsa.select_slots(layer.iq, layer.iw, layer.codes, layer.code_scales, layer.table, layer.seq_lens,
                                  layer.top, layer.page, cu_q=layer.cu, sink_blocks=1, local_blocks=2, stream=s)
    with torch.cuda.stream(s):
        ql = q[last]
    dense = qsa.paged_decode(ql, layer.kc, layer.vc, layer.table, layer.seq_lens, layer.page, stream=s)
    s.synchronize()
    for got, exp in zip((q, idx, width, dense), (want[0], want[1], want[2], want[4])):
        assert torch.equal(got, exp)


def test_wrapper_refusals_on_the_gpu():
    c = decode_case(75, [10], 8, 1, 16)
    with pytest.raises(ValueError, match="page_table"):
        qsa.paged_decode(**dict(c, page_table=c["page_table"][0]))
    with pytest.raises(ValueError, match="v_cache"):
        qsa.paged_decode(**dict(c, v_cache=c["v_cache"].float()))
    with pytest.raises(qsa.QSAError):
        qsa.paged_decode(**dict(c, q=normal(gen(76), 1, 17, 256)))
    s = select_case(77, [100], None, 4, 128, 4, 16)
    with pytest.raises(ValueError, match="multiple"):
        run_select(dict(s, page_size=18), 4)
    with pytest.raises(qsa.QSAError):
        run_select(s, 4, sink=5)
    with pytest.raises(qsa.QSAError, match="WORKSPACE"):
        run_select(s, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    r = rope_case(78, 4, 4, 1, 256, 64, 1)
    with pytest.raises(ValueError, match="sections"):
        qsa.qk_norm_rope(r["q"], r["positions"].expand(2, 4).contiguous(), r["inv_freq"])
    with pytest.raises(ValueError, match="k_cache"):
        qsa.qk_norm_rope(r["q"], r["positions"], r["inv_freq"], slots=r["positions"])


# ---- selection: rows longer than the shared memory of the choice -----------------------------

def keyed_case(score, rows, top, block=1):
    """`rows` rows of one sequence whose blocks score `score` [n] (a positive scale each, dots of 1)."""
    n = score.numel()
    page = 64 * block
    P = -(-n // 64) + 1
    g = gen(90)
    c = dict(block=block, page_size=page, cu_q=torch.tensor([0, rows], dtype=I32, device="cuda"))
    c["page_table"] = torch.randperm(P, generator=g, device="cuda").to(I32).view(1, P)
    c["seq_lens"] = torch.tensor([n * block], dtype=I32, device="cuda")
    c["q"] = torch.zeros(rows, 1, 64, dtype=BF, device="cuda")
    c["q"][:, :, 0] = 127.0
    c["weight"] = torch.ones(rows, 1, device="cuda")
    c["codes"] = torch.zeros(P * 64, 64, dtype=torch.int8, device="cuda")
    c["codes"][:, 0] = 1
    c["scales"] = torch.zeros(P * 64, device="cuda")
    j = torch.arange(n, device="cuda")
    c["scales"][c["page_table"][0, j // 64].long() * 64 + j % 64] = score
    return c


@pytest.mark.parametrize("rows", [1, 200, 1300])
@pytest.mark.parametrize("kind", ["random", "rising", "falling", "periodic", "two_values", "equal", "spread", "last"])
def test_select_order_of_a_long_row(kind, rows):
    """Scores that a sample of the row represents well, badly or not at all; one thread block per
    row of every size (few rows, more than the SMs, many)."""
    n = 40000
    x = torch.rand(n, generator=gen(91), device="cuda") + 0.5
    if kind in ("rising", "falling"):
        x = x.sort(descending=kind == "falling").values
    elif kind == "periodic":
        x[torch.arange(n, device="cuda") % 39 == 0] += 5
    elif kind == "two_values":
        x = torch.where(x > 1.3, 2.0, 1.0)
    elif kind == "equal":
        x.fill_(1.0)
    elif kind == "spread":  # over the whole range of exponents
        x = torch.exp2((x - 1) * 250)
    elif kind == "last":
        x[:-700] = 0
    c = keyed_case(x, rows, 0)
    for top, sink, local in ((512, 0, 0), (512, 1, 7), (1, 0, 0), (3000, 0, 100)):
        got, width = run_select(c, top, sink, local)
        for t in (0, rows // 2, rows - 1):
            one = dict(c, q=c["q"][t:t + 1], weight=c["weight"][t:t + 1], cu_q=None,
                       seq_lens=c["seq_lens"] - (rows - 1 - t))
            want, want_width = ref.select(one["q"], one["weight"], c["codes"], c["scales"], c["page_table"],
                                          one["seq_lens"], None, top, c["page_size"], 1, sink, local)
            assert torch.equal(got[t].cpu(), torch.from_numpy(want[0])) and int(width[t]) == int(want_width[0])


@pytest.mark.parametrize("n", [130, 500, 700])
@pytest.mark.parametrize("kind", ["random", "falling", "two_values", "equal", "spread", "few_best"])
def test_select_order_of_many_short_rows(kind, n):
    """More rows than eight per SM, none longer than 2,048 blocks."""
    x = torch.rand(n, generator=gen(92), device="cuda") + 0.5
    if kind == "falling":
        x = x.sort(descending=True).values
    elif kind == "two_values":
        x = torch.where(x > 1.2, 2.0, 1.0)
    elif kind == "equal":
        x.fill_(1.0)
    elif kind == "spread":
        x = torch.exp2((x - 1) * 250)
    elif kind == "few_best":
        x[n // 2:n // 2 + 5] += 1000
    rows = 1300
    c = keyed_case(x, rows, 0)
    c["seq_lens"] += rows
    c["page_table"] = torch.cat([c["page_table"], c["page_table"][:, :1].expand(1, 21)], 1).contiguous()
    for top, sink, local in ((100, 0, 0), (100, 1, 7), (1, 0, 0), (129, 100, 29), (500, 0, 3)):
        got, width = run_select(c, top, sink, local)
        for t in (0, 1, 2, 3, rows // 2, rows - 2, rows - 1):
            want, want_width = ref.select(c["q"][t:t + 1], c["weight"][t:t + 1], c["codes"], c["scales"], c["page_table"],
                                          c["seq_lens"] - (rows - 1 - t), None, top, c["page_size"], 1, sink, local)
            assert torch.equal(got[t].cpu(), torch.from_numpy(want[0])) and int(width[t]) == int(want_width[0])


def test_select_many_short_rows_of_several_sequences():
    c = select_case(93, [900, 3, 2003, 4500], [900, 3, 150, 270], 4, 128, 4, 64, gap=2)
    assert check_select(c, 40, 1, 3) == 0
    c["page_table"][2, 5], c["scales"][::3] = -1, float("nan")
    assert check_select(c, 40) == SLOT_RANGE
    assert check_select(c, 300) == SLOT_RANGE


def test_calls_that_read_what_the_call_before_wrote():
    """Back to back on one stream, nothing between: every call's inputs are the outputs of the one
    before it, with and without scores to compute."""
    c = select_case(94, [900, 5, 2001, 77], None, 4, 128, 4, 64)
    base = run_select(c, 40)[1]
    torch.cuda.synchronize()
    for top in (40, 600):  # 600 blocks: more than the table holds, nothing is scored
        steps, lens = [], c["seq_lens"]
        for _ in range(12):
            idx, width = run_select(dict(c, seq_lens=lens), top)
            steps.append((lens, idx, width))
            lens = width
        torch.cuda.synchronize()
        for lens, idx, width in steps:
            want = ref.select(c["q"], c["weight"], c["codes"], c["scales"], c["page_table"], lens, None, top, 64, 4, 0, 0)
            assert torch.equal(idx.cpu(), torch.from_numpy(want[0])) and torch.equal(width.cpu(), torch.from_numpy(want[1]))
    d = decode_case(95, [900, 5, 2001, 77], 16, 2, 64)
    d["seq_lens"] = run_select(c, 40)[1]  # the selection's widths as lengths
    out = qsa.paged_decode(**d)
    want, tol, _ = ref.paged_decode(d["q"], d["k_cache"], d["v_cache"], d["page_table"], base, 64, 1 / 16)
    close(out, want, tol)


def test_select_largest_budget_of_many_rows():
    """8,192 blocks of rows in thread blocks of every size."""
    x = torch.rand(30000, generator=gen(96), device="cuda") + 0.5
    for rows in (2, 160, 1200):
        c = keyed_case(x, rows, 0)
        got, width = run_select(c, 8192, 1, 50)
        for t in (0, rows - 1):
            want, want_width = ref.select(c["q"][t:t + 1], c["weight"][t:t + 1], c["codes"], c["scales"], c["page_table"],
                                          c["seq_lens"] - (rows - 1 - t), None, 8192, c["page_size"], 1, 1, 50)
            assert torch.equal(got[t].cpu(), torch.from_numpy(want[0])) and int(width[t]) == int(want_width[0])


def test_empty_page_tables_and_pools():
    c = select_case(97, [10, 20], None, 4, 128, 4, 16)
    empty = dict(c, page_table=c["page_table"][:, :0])
    assert check_select(empty, 8) == WIDTH_RANGE
    none = dict(c, codes=c["codes"][:0], scales=c["scales"][:0])
    assert check_select(none, 8) == SLOT_RANGE and check_select(none, 1) == SLOT_RANGE
    d = decode_case(98, [10, 20], 8, 1, 16)
    assert check_decode(dict(d, page_table=d["page_table"][:, :0]))[0] == WIDTH_RANGE
    assert check_decode(dict(d, k_cache=d["k_cache"][:0], v_cache=d["v_cache"][:0]))[0] == SLOT_RANGE


def test_strides_of_dimensions_of_one():
    """A single token, head or sequence may have any stride in that dimension."""
    c = decode_case(99, [300], 8, 1, 16)
    want = qsa.paged_decode(**c)
    odd = lambda t, d, n: t.as_strided(t.shape, [n if i == d else s for i, s in enumerate(t.stride())])  # noqa: E731
    got = qsa.paged_decode(**dict(c, q=odd(c["q"], 0, 3), k_cache=odd(c["k_cache"], 1, 5), v_cache=odd(c["v_cache"], 1, 1)))
    assert torch.equal(got, want)
    r = rope_case(99, 1, 1, 1, 128, 64, 1)
    want, _ = qsa.qk_norm_rope(r["q"], r["positions"], r["inv_freq"])
    got, _ = qsa.qk_norm_rope(odd(odd(r["q"], 0, 1), 1, 7), r["positions"], r["inv_freq"])
    assert torch.equal(got, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_two_calls_at_once(fp8):
    """The same inputs on two streams at the same time, each with its own outputs and workspace."""
    d = decode_case(100, [9000, 40, 3000], 16, 2, 64, fp8)
    c = select_case(101, [9000, 3000], [300, 200], 4, 128, 4, 64)
    want = qsa.paged_decode(**d), run_select(c, 100)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                got.append((qsa.paged_decode(**d), run_select(c, 100)))
    torch.cuda.synchronize()
    for out, (idx, width) in got:
        assert torch.equal(out, want[0]) and torch.equal(idx, want[1][0]) and torch.equal(width, want[1][1])


def test_stream_of_the_tensors():
    d = decode_case(102, [30], 8, 1, 16)
    assert torch.equal(qsa.paged_decode(**d, stream=torch.cuda.current_stream()), qsa.paged_decode(**d))


@pytest.mark.parametrize("Hi", [1, 4, 12, 24])
def test_select_prefill_and_decode_rows_in_one_batch(Hi):
    """Long tiles of rows beside sequences of a row or a few."""
    lens, rows = [3000] + [700, 1300, 90, 2001, 5, 900] * 2, [700] + [1, 1, 2, 1, 3, 9] * 2
    assert check_select(select_case(103, lens, rows, Hi, 128, 4, 64, gap=1), 20, 1, 2) == 0
