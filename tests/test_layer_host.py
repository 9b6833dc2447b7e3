"""Host-side tests of the layer operators (no GPU): refusals that return before any CUDA call,
the planners, the torch wrappers' checks, and the references against closed forms."""
from __future__ import annotations

import ctypes
import math

import numpy as np
import pytest
import torch

import layer_reference as ref
import top_sparse_attention_index_b200 as qsa
from top_sparse_attention_index_b200 import _binding, build_lib

A = 1 << 20  # an aligned address that is never read: every call below returns before a launch


@pytest.fixture(scope="module", autouse=True)
def lib():
    build_lib.build()
    return _binding.load_library()


def call(lib, name, order, base, **change):
    args = {**base, **change}
    return getattr(lib, name)(*[args[k] for k in order.split()])


ROPE = ("q qt qh k kt kh v vt vh qw kw off eps pos ps freq rot inter sec axes rs T Hq Hkv D qo qot qoh "
        "kd kds kdh vd vds vdh slots rows fp8 ksc vsc err stream")
ROPE_OK = dict(q=A, qt=4096, qh=256, k=A, kt=512, kh=256, v=A, vt=512, vh=256, qw=A, kw=A, off=0.0, eps=1e-6,
               pos=A, ps=0, freq=A, rot=64, inter=0, sec=None, axes=1, rs=1.0, T=0, Hq=16, Hkv=2, D=256, qo=A,
               qot=4096, qoh=256, kd=A, kds=512, kdh=256, vd=A, vds=512, vdh=256, slots=A, rows=64, fp8=0,
               ksc=1.0, vsc=1.0, err=None, stream=None)


def sections(*n):
    return (ctypes.c_int32 * len(n))(*n)


@pytest.mark.parametrize("change,status", [
    (dict(T=0), 0), (dict(T=4, Hq=0, Hkv=0), 0),
    (dict(T=-1), 1), (dict(Hq=-1), 1), (dict(rows=-1), 1),
    (dict(D=96), 2), (dict(D=512), 2), (dict(rot=24), 2), (dict(rot=272), 2), (dict(rot=-16), 2), (dict(Hq=70000), 2),
    (dict(axes=0), 1), (dict(axes=5), 1), (dict(axes=3), 1), (dict(inter=2), 1), (dict(fp8=2), 1),
    (dict(eps=-1.0), 1), (dict(eps=math.nan), 1), (dict(off=math.inf), 1), (dict(rs=math.nan), 1),
    (dict(fp8=1, ksc=0.0), 1), (dict(fp8=1, vsc=math.inf), 1),
    (dict(axes=3, sec=sections(16, 8, 9)), 1), (dict(axes=3, sec=sections(40, -4, -4)), 1),
    (dict(axes=2, sec=sections(16, 8)), 1),
    (dict(T=4, q=None), 1), (dict(T=4, qo=None), 1), (dict(T=4, k=None), 1), (dict(T=4, kd=None), 1),
    (dict(T=4, vd=None), 1), (dict(T=4, v=None), 1), (dict(T=4, pos=None), 1), (dict(T=4, freq=None), 1),
    (dict(T=65, slots=None), 1), (dict(T=4, q=A + 8), 1), (dict(T=4, qw=A + 2), 1), (dict(T=4, pos=A + 2), 1),
    (dict(T=4, qt=4100), 1), (dict(T=4, kds=-512), 1), (dict(T=4, kd=A + 8), 1), (dict(T=4, fp8=1, kd=A + 4), 1),
    (dict(T=4, fp8=1, kds=516), 1), (dict(T=4, ps=-1), 1), (dict(T=4, Hkv=0), 1),
])
def test_norm_rope_refusals(lib, change, status):
    assert call(lib, "qsa_qk_norm_rope", ROPE, ROPE_OK, **change) == status
    assert (qsa.qsa_last_error_detail() != "") == (status != 0)


PACK = "keys ks blocks n block Di S codes cs scales err stream"
PACK_OK = dict(keys=A, ks=128, blocks=A, n=0, block=4, Di=128, S=4096, codes=A, cs=128, scales=A, err=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(), 0), (dict(n=-1), 1), (dict(S=-1), 1), (dict(Di=96), 2), (dict(block=0), 1), (dict(block=17), 1),
    (dict(n=4, keys=None), 1), (dict(n=4, blocks=None), 1), (dict(n=4, codes=None), 1), (dict(n=4, scales=None), 1),
    (dict(n=4, keys=A + 8), 1), (dict(n=4, codes=A + 8), 1), (dict(n=4, scales=A + 1), 1), (dict(n=4, ks=130), 1),
    (dict(n=4, cs=136), 1), (dict(n=4, ks=-128), 1),
])
def test_pack_refusals(lib, change, status):
    assert call(lib, "qsa_pack_index_keys", PACK, PACK_OK, **change) == status
    assert (qsa.qsa_last_error_detail() != "") == (status != 0)


SELECT = ("q qt qh w ws codes cs scales table ts lens cu Tq B P pages page Hi Di block top sink local out os width "
          "work bytes err stream")
SELECT_OK = dict(q=A, qt=512, qh=128, w=A, ws=4, codes=A, cs=128, scales=A, table=A, ts=16, lens=A, cu=A, Tq=0, B=2,
                 P=16, pages=40, page=64, Hi=4, Di=128, block=4, top=64, sink=0, local=0, out=A, os=300, width=A,
                 work=A, bytes=1 << 30, err=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(), 0), (dict(Tq=0, B=0), 0),
    (dict(Tq=-1), 1), (dict(B=-1), 1), (dict(P=-1), 1), (dict(block=0), 1), (dict(block=17), 1), (dict(page=0), 1),
    (dict(page=62), 1), (dict(page=1 << 27, P=16), 2), (dict(pages=-1), 1), (dict(pages=1 << 26), 1), (dict(Di=256), 2),
    (dict(Hi=0), 2), (dict(Hi=65), 2), (dict(top=0), 1), (dict(top=2049), 1), (dict(sink=-1), 1), (dict(local=-1), 1),
    (dict(sink=33, local=32), 1), (dict(Tq=3, cu=None), 1),
    (dict(Tq=4, q=None), 1), (dict(Tq=4, w=None), 1), (dict(Tq=4, codes=None), 1), (dict(Tq=4, scales=None), 1),
    (dict(Tq=4, table=None), 1), (dict(Tq=4, lens=None), 1), (dict(Tq=4, out=None), 1), (dict(Tq=4, width=None), 1),
    (dict(Tq=4, q=A + 8), 1), (dict(Tq=4, codes=A + 8), 1), (dict(Tq=4, table=A + 2), 1), (dict(Tq=4, qt=516), 1),
    (dict(Tq=4, cs=130), 1), (dict(Tq=4, ws=-1), 1), (dict(Tq=4, os=-1), 1),
    (dict(Tq=4, work=None), 3), (dict(Tq=4, bytes=1023), 3), (dict(Tq=4, work=A + 16), 1),
])
def test_select_refusals(lib, change, status):
    assert call(lib, "qsa_select_slots", SELECT, SELECT_OK, **change) == status
    assert (qsa.qsa_last_error_detail() != "") == (status != 0)


DECODE = ("q qb qh k ks kh v vs vh table ts lens B Hq Hkv D P pages page scale fp8 ksc vsc out ob oh lse blocks work "
          "bytes err stream")
DECODE_OK = dict(q=A, qb=4096, qh=256, k=A, ks=512, kh=256, v=A, vs=512, vh=256, table=A, ts=16, lens=A, B=0, Hq=16,
                 Hkv=2, D=256, P=16, pages=40, page=64, scale=0.0625, fp8=0, ksc=1.0, vsc=1.0, out=A, ob=4096, oh=256,
                 lse=None, blocks=4, work=A, bytes=1 << 30, err=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(), 0), (dict(B=-1), 1), (dict(P=-1), 1), (dict(Hq=15), 1), (dict(Hkv=0), 1), (dict(D=128), 2),
    (dict(Hq=34), 2), (dict(page=0), 1), (dict(page=1 << 28), 2), (dict(blocks=-1), 1), (dict(blocks=65537), 1), (dict(fp8=2), 1),
    (dict(scale=math.nan), 1), (dict(fp8=1, ksc=math.inf), 1), (dict(pages=-1), 1),
    (dict(B=4, q=None), 1), (dict(B=4, k=None), 1), (dict(B=4, v=None), 1), (dict(B=4, table=None), 1),
    (dict(B=4, lens=None), 1), (dict(B=4, out=None), 1), (dict(B=4, q=A + 8), 1), (dict(B=4, k=A + 4), 1),
    (dict(B=4, lse=A + 1), 1), (dict(B=4, ks=516), 1), (dict(B=4, fp8=1, ks=520), 1), (dict(B=4, oh=-256), 1),
    (dict(B=4, work=None), 3), (dict(B=4, bytes=1000), 3), (dict(B=4, work=A + 8), 1),
])
def test_decode_refusals(lib, change, status):
    assert call(lib, "qsa_paged_decode", DECODE, DECODE_OK, **change) == status
    assert (qsa.qsa_last_error_detail() != "") == (status != 0)


@pytest.mark.parametrize("B,Hq,Hkv,P,page", [(1, 16, 2, 1, 64), (64, 24, 2, 128, 64), (1, 3, 1, 262144, 1),
                                             (4, 16, 2, 4096, 64), (300, 12, 1, 33, 100), (2, 16, 16, 0, 16)])
@pytest.mark.parametrize("request_", [0, 1, 3, 65536])
@pytest.mark.parametrize("fp8", [False, True])
def test_decode_plan(B, Hq, Hkv, P, page, request_, fp8):
    n, ws = qsa.qsa_paged_decode_plan(B, Hq, Hkv, 256, P, page, fp8, 148, request_)
    # a block per KV head in every group; no group without a unit of tokens at the sequences'
    # greatest length
    assert n % Hkv == 0 and Hkv <= n <= Hkv * max(1, B * -(-P * page // (64 if fp8 else 32)))
    if request_:
        assert n <= max(request_, Hkv)
    assert ws == 0 if n == Hkv else ws >= n * 2 * (Hq // Hkv) * 257 * 4
    # a plan asked for again by its own count is itself (a caller sizes its workspace with it)
    assert qsa.qsa_paged_decode_plan(B, Hq, Hkv, 256, P, page, fp8, 148, n) == (n, ws)


def test_select_workspace_is_bounded():
    assert qsa.qsa_select_slots_workspace_bytes(0, 4, 16, 64, 4, 128, 4) == 0
    assert qsa.qsa_select_slots_workspace_bytes(1, 1, 16, 64, 4, 128, 4) == 256 * 4
    # scores of a chunk of rows: 512 MiB while 64 rows fit; codes and gains of 256 columns per tile of rows
    n = qsa.qsa_select_slots_workspace_bytes(1 << 16, 1, 1024, 64, 4, 128, 4)
    tiles = 8 * (8192 // 64 + 1)
    assert n == (512 << 20) + (tiles * 16 + 255) // 256 * 256 + tiles * 256 * 132
    for bad in ((1, 1, 16, 62, 4, 128, 4), (1, 1, 16, 64, 0, 128, 4), (1, 1, 16, 64, 4, 96, 4)):
        with pytest.raises(qsa.QSAError):
            qsa.qsa_select_slots_workspace_bytes(*bad)


def test_wrappers_refuse_cpu_tensors_and_bad_shapes():
    bf, i32 = torch.bfloat16, torch.int32
    q = torch.zeros(2, 4, 128, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.qk_norm_rope(q, torch.zeros(2, dtype=i32), torch.zeros(32))
    with pytest.raises(ValueError, match="CUDA"):
        qsa.pack_index_keys(torch.zeros(8, 128, dtype=bf), torch.zeros(1, dtype=i32),
                            torch.zeros(2, 128, dtype=torch.int8), torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        qsa.select_slots(q, torch.zeros(2, 4), torch.zeros(2, 128, dtype=torch.int8), torch.zeros(2),
                         torch.zeros(2, 1, dtype=i32), torch.zeros(2, dtype=i32), 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        qsa.paged_decode(torch.zeros(2, 4, 256, dtype=bf), torch.zeros(8, 2, 256, dtype=bf),
                         torch.zeros(8, 2, 256, dtype=bf), torch.zeros(2, 1, dtype=i32), torch.zeros(2, dtype=i32), 8)


# ---- the references against closed forms ------------------------------------------------------

def test_reference_rotation_turns_by_the_angle():
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    x[..., 0], x[..., 9] = 3.0, 4.0
    freq = torch.tensor([math.pi / 2] + [0.0] * 15)
    y, _ = ref.norm_rope(x, None, 0.0, 0.0, torch.tensor([3]), freq, None, False, 2.0)
    # three quarter turns of (3, 0): (0, -3), times the scale; dimension 9 turns by 0
    assert torch.allclose(y[0, 0, [0, 16]], torch.tensor([0.0, -6.0], dtype=torch.float64), atol=1e-6)
    assert y[0, 0, 9] == 8.0
    y, _ = ref.norm_rope(x, torch.ones(64, dtype=torch.bfloat16), 0.0, 0.0, torch.tensor([0]), freq, None, True, 1.0)
    assert torch.allclose(y[0, 0, 0], torch.tensor(3.0 / math.sqrt(25.0 / 64.0), dtype=torch.float64))


def test_reference_codes():
    codes, scale = ref.codes_of(np.array([[127.0, -63.5, 0.5, 1.5], [0, 0, 0, 0], [np.inf, 1, 0, 0]], np.float32))
    assert codes.tolist() == [[127, -64, 0, 2], [0, 0, 0, 0], [0, 0, 0, 0]]  # halves to even
    assert scale[0] == 1.0 and scale[1] == 0.0 and np.isnan(scale[2])


def test_reference_selection():
    # one head, keys along one axis: the scores are the codes; equal ones go to the lower block
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    q[..., 0] = 127.0
    codes = torch.zeros(8, 64, dtype=torch.int8)
    codes[:, 0] = torch.tensor([5, 9, -3, 9, 1, 7, 0, 0])
    table = torch.tensor([[1, 0]], dtype=torch.int32)  # 4 blocks of 2 slots per page of 8
    got, width = ref.select(q, torch.ones(1, 1), codes, torch.ones(8), table, torch.tensor([15]), None, 2, 8, 2, 0, 0)
    # logical scores: 1 7 0 0 | 5 9 -> 0 (of -3), 7 complete blocks; best are logical 5 (9) and 1 (7)
    assert got.tolist() == [[10, 11, 2, 3, 6]] and width.tolist() == [5]
    got, _ = ref.select(q, torch.ones(1, 1), codes, torch.ones(8), table, torch.tensor([15]), None, 3, 8, 2, 1, 1)
    assert got.tolist() == [[8, 9, 2, 3, 4, 5, 6]]


def test_reference_attention_of_equal_keys_is_the_mean():
    k = torch.zeros(8, 1, 256, dtype=torch.bfloat16)
    v = torch.arange(8.0)[:, None, None].expand(8, 1, 256).to(torch.bfloat16)
    q = torch.ones(2, 2, 256, dtype=torch.bfloat16)
    table = torch.tensor([[3, 0], [-1, 9]], dtype=torch.int32)
    out, _, lse = ref.paged_decode(q, k, v, table, torch.tensor([3, 4]), 2, 1 / 16)
    assert torch.allclose(out[0], torch.full((2, 256), (6 + 7 + 0) / 3, dtype=torch.float64))
    assert torch.allclose(lse[0], torch.full((2,), math.log2(3), dtype=torch.float64))
    assert (out[1] == 0).all() and torch.isinf(lse[1]).all()
