"""The layer operators where rounding, memory order or a failing wait decides the result:
calls that follow each other without a pause, scores a step apart, exact counts of slots."""
from __future__ import annotations

import pytest
import torch

import layer_reference as ref
import top_sparse_attention_index_b200 as qsa
from test_layer_gpu import BF, F8, I32, err_word, gen, normal

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
