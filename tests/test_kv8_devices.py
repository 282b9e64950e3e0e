"""Calls over the 8-bit cache refuse tensors on different GPUs, and closed objects, before they reach the library
(stand-ins for tensors: no GPU needed)."""

import numpy as np
import pytest
import torch

from invariant_vd_step_gb300 import vd
from test_tree_devices import OnGpu


def plan_without_library(monkeypatch):
    class NoLibrary:
        def __getattr__(self, name):
            def call(*a):
                raise AssertionError(f"{name} reached")
            return call
    monkeypatch.setattr(vd, "lib", NoLibrary)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(vd, "_current_raw_stream", lambda device: 0)
    plan = object.__new__(vd.KV8Plan)
    spec = type("Spec", (), dict(n_heads=4, head_dim=64, qkv_dim=512, vocab=100))
    plan.h, plan.model = 1, type("M", (), dict(h=1, spec=spec))()
    plan.num_tokens, plan.num_logit_rows = 3, 3
    other = lambda h=1: type("P", (), dict(h=h, model=plan.model))()  # noqa: E731
    return plan, other


def refused(calls):
    for i, call in enumerate(calls):
        with pytest.raises(vd.VDError) as e:
            call()
            pytest.fail(f"call {i} was taken")
        assert e.value.code == vd.VD_ERR_INVALID_ARG


def test_tensors_on_two_gpus_are_refused(monkeypatch):
    plan, other = plan_without_library(monkeypatch)
    q = [OnGpu((3, 4, 64), torch.bfloat16, d) for d in (0, 1)]
    qkv = [OnGpu((3, 512), torch.bfloat16, d) for d in (0, 1)]
    try:
        refused([lambda: plan.attention(other(), other(), 0, q[1], q[0]),
                 lambda: plan.attention(other(), other(), 0, q[0], q[1]),
                 lambda: plan.attention(other(), other(), 0, q[1], q[1]),  # not the current device
                 lambda: plan.rope_kv(other(), other(), 0, qkv[1], q[0]),
                 lambda: plan.rope_kv(other(), other(), 0, qkv[0], q[1]),
                 lambda: plan.step(other(), other(), OnGpu((3, 100), torch.float32, 1))])
    finally:
        plan.h = None  # nothing for close() to destroy


def test_closed_objects_are_refused(monkeypatch):
    plan, other = plan_without_library(monkeypatch)
    q = OnGpu((3, 4, 64), torch.bfloat16, 0)
    try:
        refused([lambda: plan.attention(other(None), other(), 0, q, OnGpu((3, 4, 64), torch.bfloat16, 0)),
                 lambda: plan.attention(other(), other(None), 0, q, OnGpu((3, 4, 64), torch.bfloat16, 0)),
                 lambda: plan.seal(other(None), other(), 0), lambda: plan.seal(other(), other(None), 0)])
        plan.model.h = None
        refused([lambda: plan.seal(other(), other(), 0)])
    finally:
        plan.h = None


def test_a_pools_view_is_the_memory_whatever_mode_it_was_made_in():
    spec = type("Spec", (), dict(n_layers=2, n_kv_heads=1, head_dim=64))
    pool = object.__new__(vd.KVPool)
    pool.h, pool._pages, pool.num_pages, pool.model = None, None, 3, type("M", (), dict(spec=spec))()
    pool.memory = torch.zeros(2 * 3 * 2 * 16 * 64 * 2 + 256, dtype=torch.uint8)
    with torch.inference_mode():
        assert pool.view().shape == (2, 3, 2, 1, 16, 64)
    x = torch.ones(64, requires_grad=True)
    (pool.view() * x).sum().backward()  # (refused for tensors of inference mode)
    a, b = pool.view(), pool.view()
    a[1, 2, 0, 0, 5, 7] = 3.0
    assert b[1, 2, 0, 0, 5, 7] == 3.0 and a is not b
    np.testing.assert_array_equal(pool.memory[:-256].view(torch.bfloat16).float().numpy().nonzero()[0],
                                  [((1 * 3 + 2) * 2 * 16 + 5) * 64 + 7])
    pool.memory = torch.zeros_like(pool.memory)  # other memory: another view
    assert (pool.view() == 0).all()
    pool.memory = None
    with pytest.raises(RuntimeError):
        pool.view()


def test_numbers_that_32_bits_do_not_hold_are_refused(monkeypatch):
    plan, other = plan_without_library(monkeypatch)
    good = dict(cu_q=[0, 1], cached_len=[3], page_table=[[0]], open_table=[[0]], token_ids=[1], logit_rows=[0])
    try:
        refused([lambda k=k, v=v: plan.plan(other(), other(), **{**good, k: v}) for k, v in [
            ("cu_q", [0, 2 ** 32 + 1]), ("cached_len", [2 ** 32]), ("page_table", [[2 ** 32]]), ("open_table", [[-2 ** 32]]),
            ("open_table", [[0.0]]), ("token_ids", [2 ** 32 + 1]), ("logit_rows", [2 ** 32])]])
        with pytest.raises(AssertionError, match="reached"):
            plan.plan(other(), other(), **good)
    finally:
        plan.h = None


def test_page_ids_stay_alive_until_the_call():
    class Passing:  # an array of ids that nothing else holds, and that may not be written
        def __array__(self, dtype=None, copy=None):
            a = np.arange(5, dtype=np.int32)
            a.flags.writeable = False
            return a
    a = vd._ids(Passing())
    assert a.flags.writeable and a.tolist() == [0, 1, 2, 3, 4]
    n, src, dst = vd._page_lists(Passing(), [4, 3, 2, 1, 0])
    assert n == 5
    kept = np.frombuffer((vd.ctypes.c_int32 * 5).from_address(vd.ctypes.addressof(src)), np.int32)
    assert kept.tolist() == [0, 1, 2, 3, 4]


def test_read_only_page_ids_are_read_while_they_live(monkeypatch):
    """Read-only arrays that nothing else holds, passed to each call that takes page ids: what the library reads at the
    address that it gets is those ids, with other arrays of the size made in between."""
    import ctypes
    junk, seen = [], []

    class Library:
        def __getattr__(self, name):
            def call(*a):
                n, src, dst = a[-4:-1]
                junk.extend(np.full(n, -1, np.int32) for _ in range(50))  # takes up memory that is free
                at = lambda p: p if isinstance(p, int) else ctypes.addressof(p)  # noqa: E731
                seen.append([np.frombuffer((ctypes.c_int32 * n).from_address(at(p)), np.int32).tolist()
                             for p in (src, dst)])
                return 0
            return call
    monkeypatch.setattr(vd, "lib", Library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(vd, "_current_raw_stream", lambda device: 0)
    model = type("M", (), dict(h=1))()
    cache, pool = object.__new__(vd.KV8Cache), object.__new__(vd.KVPool)
    cache.h = pool.h = 1
    cache.model = pool.model = model

    def ids(first):
        a = np.arange(first, first + 700, dtype=np.int32)
        a.flags.writeable = False
        return a
    try:
        for call in (pool.copy_pages, cache.copy_pages, lambda s, d: cache.seal(pool, s, d),
                     lambda s, d: cache.unseal(pool, s, d)):
            call(ids(0), ids(1000))
            assert seen.pop() == [list(range(700)), list(range(1000, 1700))]
            call(np.broadcast_to(np.int32(5), 3), ids(7)[:3])  # read-only views
            assert seen.pop() == [[5, 5, 5], [7, 8, 9]]
    finally:
        cache.h = pool.h = None


def test_page_tables_that_are_not_rows_of_the_requests_are_refused(monkeypatch):
    plan, other = plan_without_library(monkeypatch)
    good = dict(cu_q=[0, 1, 2], cached_len=[3, 4], page_table=[[0], [1]], open_table=[[0], [1]])
    none = dict(cu_q=[0], cached_len=[], page_table=[], open_table=[])
    try:
        refused([lambda k=k, v=v, g=g: plan.plan(other(), other(), **{**g, k: v}) for g, k, v in [
            (good, "page_table", [0, 1, 2]), (good, "open_table", np.zeros((3, 1), int)), (none, "page_table", [[1]]),
            (none, "open_table", [0]), (good, "cu_q", [0, 1]), (none, "cu_q", [])]])
        for g in (good, none):
            with pytest.raises(AssertionError, match="reached"):
                plan.plan(other(), other(), **g)
    finally:
        plan.h = None
