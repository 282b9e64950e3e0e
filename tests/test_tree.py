"""Token trees on the host: refusals that come before any CUDA call."""

import ctypes

import pytest

from invariant_vd_step_gb300 import build, vd


def test_tree_calls_refuse_null_handles():
    build.build()
    L, out, b = vd.lib(), ctypes.c_void_p(), vd.TreeBatch()
    assert L.vd_tree_create(None, 8, ctypes.byref(out)) == vd.VD_ERR_INVALID_ARG
    assert not out.value
    assert L.vd_tree_plan(None, None, ctypes.byref(b), None) == vd.VD_ERR_INVALID_ARG
    assert L.vd_op_tree_attention(None, None, 0, 64, 64, None) == vd.VD_ERR_INVALID_ARG
    assert L.vd_op_tree_rope_kv(None, None, 0, 64, 64, None) == vd.VD_ERR_INVALID_ARG
    assert L.vd_step_tree(None, None, 64, None) == vd.VD_ERR_INVALID_ARG
    assert L.vd_tree_accept(None, None, None, 64, 64, 64, 8, None) == vd.VD_ERR_INVALID_ARG
    L.vd_destroy_tree(None)  # nothing to do


def test_a_closed_tree_or_model_is_refused():
    tree = object.__new__(vd.Tree)
    tree.h, tree.model = None, type("M", (), {"h": 1})()
    with pytest.raises(vd.VDError):
        tree._live()
    tree.h, tree.model.h = 1, None
    with pytest.raises(vd.VDError):
        tree._live()
    tree.h = None  # nothing for close() to destroy
