"""The drafted-tree operators' binding and library on the host: refusals and
loading beside those of test_tree_ops.py."""
import ctypes

import pytest

from decode_megakernel_llama_gb300 import _lib
from decode_megakernel_llama_gb300.build import build
from test_tree_ops import tree_args


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def test_a_negative_limit_of_waits_is_refused(lib):
    a = tree_args(wait_ns=-1)
    assert lib.mk_tree_attention(ctypes.byref(a), None) == _lib.MK_ERR_INVALID_ARG
    assert b"wait_ns" in lib.mk_last_error()


def test_the_binding_has_the_headers_numbers():
    text = open(_lib.HEADER).read()
    for name in ("MK_MAX_TREE", "MK_F32", "MK_BF16"):
        assert f"#define {name} {getattr(_lib, name)}" in text, name
