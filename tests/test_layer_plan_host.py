"""The selection's workspace over many shapes (no GPU): what the header says it may come to."""
from __future__ import annotations

import random

import pytest

import top_sparse_attention_index_b200 as qsa
from top_sparse_attention_index_b200 import build_lib

MIB = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_lib.build()


def bound(Tq, B, P, page, Hi, Di, block):
    """Scores: 512 MiB, or 64 rows where those are more, in chunks of rows as equal as can be.  Codes
    and gains of all rows in tiles of 256 columns (heads rounded up to a power of two), and in
    every chunk a tile more for each of its sequences at most."""
    ld = -(-P * (page // block) // 32) * 32
    if Tq == 0 or ld == 0:
        return 0
    heads = 1 << (Hi - 1).bit_length()
    rows = min(max(512 * MIB // (4 * ld), 64), (2 ** 30 - 1) // ld)
    chunks = -(-Tq // rows)
    scores = min(Tq, rows) * ld * 4 + 256
    if heads > 32 or Tq * heads * 2 <= B * 256:
        return scores
    tile = 256 * (Di + 4) + 16
    return scores + ((Tq + chunks) * heads // 256 + chunks * min(B, rows, Tq)) * tile + 256


def test_select_workspace_of_random_shapes():
    rng = random.Random(5)
    for _ in range(5000):
        block = rng.choice((1, 2, 3, 4, 8, 16))
        page = block * rng.choice((1, 3, 16, 64, 256))
        P = int(2 ** rng.uniform(0, 28)) // page + 1
        Tq, B = int(2 ** rng.uniform(0, 18)), int(2 ** rng.uniform(0, 12))
        shape = (Tq, B, P, page, rng.randint(1, 64), rng.choice((64, 128)), block)
        n = qsa.qsa_select_slots_workspace_bytes(*shape)
        assert 0 < n <= bound(*shape), shape


def test_select_workspace_of_the_largest_shapes():
    # 64 rows over 2^23 blocks: more than 512 MiB of scores, all the same one chunk
    assert qsa.qsa_select_slots_workspace_bytes(64, 1, 1 << 19, 64, 4, 128, 4) <= (2 << 30) + (2 << 20)
    # many heads of many rows: their codes are the larger part
    n = qsa.qsa_select_slots_workspace_bytes(262144, 1, 16, 64, 32, 128, 4)
    assert 262144 * 32 * 132 < n - 262144 * 256 * 4 < 262144 * 32 * 132 * 1.01
    # many sequences: a tile more for each in every chunk
    one, many = (qsa.qsa_select_slots_workspace_bytes(65536, B, 256, 64, 16, 128, 4) for B in (1, 2048))
    chunks = -(-65536 * 4096 * 4 // (512 * MIB))
    assert many - one <= chunks * 2048 * (256 * 132 + 16)
