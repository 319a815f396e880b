"""What the operators of pages write must overlap nothing that they read: refused on the host, before any CUDA call; and what
is not an overlap is not refused (the call then goes as far as the GPU, or does nothing for no tokens)."""
import ctypes

import pytest

from decode_megakernel_llama_gb300 import _lib
from tests.test_paged import FAKE, FAR, Q8, lib, pages_args, paged_args, rope_args  # noqa: F401  (lib: the fixture)

OUT = 40 * 512 * 2  # bytes of out
TABLE, STARTS, LENGTHS = 7 * FAR, 7 * FAR + 4096, 7 * FAR + 8192


def _paged(**kw):
    a = dict(table=TABLE, starts=STARTS, lengths=LENGTHS)
    a.update(kw)
    return paged_args(**a)


@pytest.mark.parametrize("bad", [
    dict(table=FAR), dict(table=FAR + OUT - 4), dict(table=FAR - 3 * 8 * 4 + 4), dict(starts=FAR + 512), dict(starts=FAR - 12),
    dict(lengths=FAR + 1024), dict(status=FAR + OUT - 4), dict(status=LENGTHS + 8), dict(status=TABLE), dict(status=FAKE + 64),
    dict(status=2 * FAKE), dict(status=3 * FAKE + 16), dict(status=5 * FAKE, **Q8), dict(status=STARTS + 12),
    dict(workspace=FAR, workspace_bytes=64), dict(workspace=FAR - 64, workspace_bytes=80), dict(workspace=FAKE, workspace_bytes=16),
    dict(workspace=2 * FAKE + 4096, workspace_bytes=16), dict(workspace=3 * FAKE - 16, workspace_bytes=32),
    dict(workspace=6 * FAKE, workspace_bytes=16, **Q8), dict(workspace=TABLE, workspace_bytes=16),
    dict(workspace=STARTS, workspace_bytes=16), dict(workspace=LENGTHS - 16, workspace_bytes=32),
    dict(workspace=8 * FAR, workspace_bytes=64, status=8 * FAR + 60),
])
def test_attention_refuses(lib, bad):  # noqa: F811
    assert lib.mk_paged_attention(ctypes.byref(_paged(**bad)), None) == -1
    assert b"overlaps" in lib.mk_last_error()


@pytest.mark.parametrize("kw", [
    dict(), dict(status=FAR + OUT), dict(status=FAR - 4), dict(workspace=FAR + OUT, workspace_bytes=64), dict(status=LENGTHS + 12),
    dict(workspace=8 * FAR, workspace_bytes=64, status=8 * FAR + 64), dict(workspace=2 * FAKE, workspace_bytes=0),
    dict(out_stride=1024, status=FAR + 1024), dict(out_stride=1024, table=FAR + 1024),  # (in the gaps between out's rows)
])
def test_attention_does_not_refuse(lib, kw):  # noqa: F811
    rc = lib.mk_paged_attention_workspace(ctypes.byref(_paged(**kw)))  # (checks alike; follows no pointer)
    assert rc >= 0 or b"overlaps" not in lib.mk_last_error()


ROPE = dict(positions=7 * FAR, rows=7 * FAR + 64, inv_freq=7 * FAR + 128)  # n = 4, rot = 64; rows of 256 fp32 queries


@pytest.mark.parametrize("bad,word", [
    (dict(positions=2 * FAKE + 16), b"overlaps"), (dict(rows=2 * FAKE + 1020), b"overlaps"), (dict(inv_freq=2 * FAKE - 248), b"overlaps"),
    (dict(slot_of=3 * FAKE), b"overlaps"), (dict(q_norm=4 * FAKE + 8), b"overlaps"), (dict(k_norm=2 * FAKE), b"overlaps"),
    (dict(q_stride=512, positions=2 * FAKE + 1020), b"overlaps"), (dict(q_stride=512, positions=2 * FAKE + 2048 - 12), b"overlaps"),
])
def test_rope_append_refuses(lib, bad, word):  # noqa: F811
    a = rope_args(**{**ROPE, **bad})
    assert lib.mk_rope_append(ctypes.byref(a), None) == -1 and word in lib.mk_last_error()
    assert lib.mk_rope_append_e4m3(ctypes.byref(a), 9 * FAR, 10 * FAR, None) == -1 and word in lib.mk_last_error()


@pytest.mark.parametrize("bad", [dict(positions=9 * FAR + 4), dict(rows=10 * FAR), dict(inv_freq=9 * FAR - 8), dict(q_norm=10 * FAR + 64)])
def test_rope_append_e4m3_refuses_scales_on_what_it_reads(lib, bad):  # noqa: F811
    assert lib.mk_rope_append_e4m3(ctypes.byref(rope_args(**{**ROPE, **bad})), 9 * FAR, 10 * FAR, None) == -1
    assert b"overlaps" in lib.mk_last_error()


@pytest.mark.parametrize("write", [True, False])
@pytest.mark.parametrize("name", ["table", "lengths", "first", "slot_of"])
def test_moves_refuse_index_arrays_in_what_they_write(lib, name, write):  # noqa: F811
    a = dict(table=7 * FAR, lengths=8 * FAR)
    for at in ((3 * FAKE + 64, 4 * FAKE) if write else (FAKE, 2 * FAKE + 1024)):
        args = pages_args(**{**a, name: at})
        assert getattr(lib, "mk_kv_write_pages" if write else "mk_kv_read_pages")(ctypes.byref(args), None) == -1
        assert b"overlaps table" in lib.mk_last_error()
    if write:
        args = pages_args(**{**a, "cache_dtype": 2, "k_scales": 9 * FAR, "v_scales": 10 * FAR, name: 10 * FAR + 16})
        assert lib.mk_kv_write_pages(ctypes.byref(args), None) == -1
        assert b"overlaps table" in lib.mk_last_error()


def test_rows_with_gaps():
    """meet_rows, as the refusals use it: every place of a small range against rows of 3 bytes, 5 apart."""
    rows = {5 * r + b for r in range(3) for b in range(3)}

    def meets(y, size, n=3, step=5, row=3):
        if y <= 0:
            return -y < size
        k, at = divmod(y, step)
        return k < n and (at < row or (k + 1 < n and size > step - at))
    for y in range(-9, 20):
        for size in range(1, 12):
            assert meets(y, size) == bool(rows & set(range(y, y + size)))
