"""Refusals of the paged-cache and packed-attention entry points (CPU only: every
call here is refused on the host, before any launch), and the plain forms that the
GPU tests compare with."""
import ctypes

import pytest
import torch

import paged_util as U
from decode_attention_kivi_b200 import _native as N
from decode_attention_kivi_b200 import build as B

FAKE = 1 << 20  # an aligned address that no refused call touches
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.lib()


def _workspace(lib, hkv, hq, dim):
    n = ctypes.c_size_t()
    return N.STATUS[lib.kivi_attention_workspace_bytes(hkv, hq, dim, ctypes.byref(n))], n.value


def test_workspace_bytes(lib):
    st, n = _workspace(lib, 8, 32, 128)
    assert st == "KIVI_OK" and n >= 256
    for hkv, hq, dim in [(8, 20, 128), (8, 8, 96), (1, 256, 64)]:
        assert _workspace(lib, hkv, hq, dim)[0] == "KIVI_ERR_UNSUPPORTED"
    assert _workspace(lib, 0, 8, 128)[0] == "KIVI_ERR_INVALID_ARG"
    assert N.STATUS[lib.kivi_attention_workspace_bytes(8, 8, 128, None)] == "KIVI_ERR_INVALID_ARG"


ASSIGN = dict(lengths=FAKE, new=FAKE, batch=4, table=FAKE, width=8, free=FAKE, num_free=FAKE,
              pages=32, page=16, kv=FAKE, num_free_out=FAKE, offsets=FAKE, slots=FAKE,
              positions=FAKE, rows=10, status=FAKE, stream=None)


@pytest.mark.parametrize("change,want", [
    ({"page": 24}, "UNSUPPORTED"), ({"page": 8}, "UNSUPPORTED"), ({"page": 512}, "UNSUPPORTED"),
    ({"page": 0}, "INVALID_ARG"), ({"batch": 0}, "INVALID_ARG"), ({"batch": 4097}, "UNSUPPORTED"),
    ({"width": 0}, "INVALID_ARG"), ({"rows": -1}, "INVALID_ARG"), ({"pages": 0}, "INVALID_ARG"),
    ({"pages": 1 << 27}, "INVALID_ARG"), ({"width": 1 << 27}, "INVALID_ARG"),
    ({"lengths": None}, "INVALID_ARG"), ({"slots": None}, "INVALID_ARG"),
    ({"offsets": FAKE + 2}, "INVALID_ARG"), ({"status": None}, "INVALID_ARG"),
    ({"num_free": None}, "INVALID_ARG"),
])
def test_assign_refusals(lib, change, want):
    a = {**ASSIGN, **change}
    assert N.STATUS[lib.kivi_paged_assign(*a.values())] == "KIVI_ERR_" + want


APPEND = dict(k=FAKE, ks=1024, v=FAKE, vs=1024, slots=FAKE, rows=4, kp=FAKE, vp=FAKE, pages=8,
              page=16, hkv=8, dim=128, status=None, stream=None)


@pytest.mark.parametrize("change,want", [
    ({"dim": 96}, "UNSUPPORTED"), ({"page": 20}, "UNSUPPORTED"), ({"hkv": 0}, "INVALID_ARG"),
    ({"ks": 1020}, "INVALID_ARG"), ({"vs": 1016}, "INVALID_ARG"), ({"k": FAKE + 8}, "INVALID_ARG"),
    ({"vp": None}, "INVALID_ARG"), ({"rows": -1}, "INVALID_ARG"), ({"slots": None}, "INVALID_ARG"),
    ({"status": FAKE + 1}, "INVALID_ARG"),
])
def test_append_refusals(lib, change, want):
    a = {**APPEND, **change}
    assert N.STATUS[lib.kivi_paged_append(*a.values())] == "KIVI_ERR_" + want


def test_append_of_no_rows_is_a_no_op(lib):
    assert lib.kivi_paged_append(*{**APPEND, "rows": 0, "k": None, "v": None}.values()) == 0


PACKED = dict(q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, out=FAKE, os=4096, dtype=0,
              offsets=FAKE, batch=2, rows=10, hkv=8, hq=32, dim=128, scale=0.0, ws=FAKE,
              wsb=BIG, stream=None)
PAGED = dict(q=FAKE, qs=4096, kp=FAKE, vp=FAKE, out=FAKE, os=4096, dtype=0, table=FAKE, width=4,
             kv=FAKE, offsets=FAKE, batch=2, rows=10, max_new=1, pages=8, page=16, hkv=8, hq=32,
             dim=128, scale=0.0, ws=FAKE, wsb=BIG, stream=None)
BOTH = [
    ({"dtype": 2}, "UNSUPPORTED"), ({"dim": 80}, "UNSUPPORTED"), ({"hq": 30}, "UNSUPPORTED"),
    ({"batch": 0}, "INVALID_ARG"), ({"batch": 4097}, "UNSUPPORTED"), ({"rows": -1}, "INVALID_ARG"),
    ({"scale": float("nan")}, "INVALID_ARG"), ({"q": FAKE + 8}, "INVALID_ARG"),
    ({"out": None}, "INVALID_ARG"), ({"qs": 4090}, "INVALID_ARG"), ({"os": 4088}, "INVALID_ARG"),
    ({"offsets": None}, "INVALID_ARG"), ({"ws": None}, "INVALID_ARG"),
    ({"wsb": 16}, "BUFFER_TOO_SMALL"), ({"rows": 1 << 27}, "INVALID_ARG"),
]


@pytest.mark.parametrize("change,want", BOTH + [
    ({"k": None}, "INVALID_ARG"), ({"vs": 1000}, "INVALID_ARG"), ({"ks": 1028}, "INVALID_ARG")])
def test_packed_refusals(lib, change, want):
    a = {**PACKED, **change}
    assert N.STATUS[lib.kivi_packed_attention(*a.values())] == "KIVI_ERR_" + want


@pytest.mark.parametrize("change,want", BOTH + [
    ({"page": 48}, "UNSUPPORTED"), ({"max_new": 0}, "INVALID_ARG"), ({"kp": None}, "INVALID_ARG"),
    ({"table": None}, "INVALID_ARG"), ({"kv": FAKE + 2}, "INVALID_ARG"),
    ({"width": 0}, "INVALID_ARG"), ({"pages": 1 << 25}, "INVALID_ARG")])
def test_paged_refusals(lib, change, want):
    a = {**PAGED, **change}
    assert N.STATUS[lib.kivi_paged_attention(*a.values())] == "KIVI_ERR_" + want


def test_attention_of_no_rows_is_a_no_op(lib):
    assert lib.kivi_packed_attention(*{**PACKED, "rows": 0, "q": None}.values()) == 0
    assert lib.kivi_paged_attention(*{**PAGED, "rows": 0, "q": None}.values()) == 0


def test_attention_status_needs_a_workspace(lib):
    assert N.STATUS[lib.kivi_attention_status(None, None, None)] == "KIVI_ERR_INVALID_ARG"


def test_binding_refuses_host_tensors_and_other_objects():
    import decode_attention_kivi_b200 as K

    z = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    n, ws = torch.zeros(2, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        K.kivi_packed_attention(z, z, z, n, ws)
    with pytest.raises(ValueError, match="CUDA"):
        K.kivi_paged_attention(z, z[None], z[None], n[None], n, n, ws)
    with pytest.raises(ValueError, match="CUDA"):
        K.kivi_paged_append(z, z, n, z[None], z[None])
    with pytest.raises(ValueError, match="CUDA"):
        K.kivi_paged_assign(n, n, n[None], n, n, 16, kv_lengths=n, num_free_out=n, offsets=n,
                            slots=n, positions=n, status=n)
    with pytest.raises(TypeError, match="q must be a tensor"):
        K.kivi_packed_attention([1.0], z, z, n, ws)
    with pytest.raises(TypeError, match="block_table must be a tensor"):
        K.kivi_paged_assign(n, n, None, n, n, 16, kv_lengths=n, num_free_out=n, offsets=n,
                            slots=n, positions=n, status=n)
    with pytest.raises(TypeError, match="arguments"):
        N.binding().append(z, z)


# ---- the plain forms ----

def test_plain_attention_by_hand():
    """Two rows, the last of three keys: weights 1/2, 1/2 and then 1/4, 1/4, 1/2 at sm_scale ln 2."""
    import math

    q = torch.tensor([[[1.0]], [[1.0]]])
    k = torch.tensor([[[0.0]], [[0.0]], [[1.0]]])
    v = torch.tensor([[[1.0]], [[-3.0]], [[8.0]]])
    out, mean = U.attend(q, k, v, sm_scale=math.log(2))
    assert out.flatten().tolist() == pytest.approx([-1.0, 3.5])
    assert mean.flatten().tolist() == pytest.approx([2.0, 5.0])
    # a request with fewer keys than rows: its first rows see none
    out, mean = U.attend(torch.ones(3, 1, 1), k[:1], v[:1])
    assert out.flatten().tolist() == [0.0, 0.0, 1.0]


def test_books_by_hand():
    b = U.Books([3, 5, 0], [[7, 0], [1, 2], [0, 0]], [9, 8, 6, 0, 0], 3, 4)
    offsets, slots, positions, status = b.step([2, -1, 5], 8)
    # pages 1 and 2 are pushed on 9, 8, 6; then 2 goes to request 0, 1 and 6 to request 2
    assert status == 0 and offsets == [0, 2, 2, 7] and b.lengths == [5, 0, 5]
    assert b.table[0] == [7, 2] and b.table[2] == [1, 6] and b.num_free == 2
    assert slots == [31, 8, 4, 5, 6, 7, 24, -1] and positions == [3, 4, 0, 1, 2, 3, 4, 0]
    assert b.step([4, 0, 0], 8)[3] == 4 and b.lengths == [5, 0, 5]     # past the table's width
    assert b.step([0, 8, 3], 8)[3] == 4                                 # more rows than there are
    b.num_free = 1
    assert b.step([0, 8, 0], 8) == ([0] * 4, [-1] * 8, [0] * 8, 8)      # not enough pages


def test_paged_attention_without_rows_takes_a_max_new_of_zero(lib):
    """The largest number of new rows of a step that has none."""
    a = {**PAGED, "rows": 0, "q": None, "out": None, "max_new": 0}
    assert lib.kivi_paged_attention(*a.values()) == 0
    assert N.STATUS[lib.kivi_paged_attention(*{**a, "max_new": -1}.values())] == "KIVI_ERR_INVALID_ARG"


# ---- the binding's build ----

def test_a_binding_for_another_torch_is_built_again(lib, monkeypatch, tmp_path):
    """With nothing newer among the sources: another torch alone makes it stale."""
    assert not B.binding_stale()
    ran = []
    with monkeypatch.context() as m:
        m.setattr(B, "binding_target", lambda: "torch 0.1, Python 3.0")
        m.setattr(B, "BINDING_TARGET", str(tmp_path / "_build" / "target"))
        m.setattr(B.os, "replace", lambda a, b: None)
        m.setattr(B.subprocess, "run", lambda cmd, check: ran.append(cmd))
        B.build_binding()
        assert len(ran) == 1 and any("torch 0.1" in a for a in ran[0])
        B.build_binding()
        assert len(ran) == 1
    assert not B.binding_stale()


def test_a_binding_for_another_torch_is_refused(lib, monkeypatch):
    monkeypatch.setattr(N, "_binding", None)
    monkeypatch.setattr(B, "binding_target", lambda: "torch 0.1, Python 3.0")
    with pytest.raises(RuntimeError, match="built for torch"):
        N.binding()
