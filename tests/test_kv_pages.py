"""vd_pages: reference counts, forks and compaction of pages (host logic, no GPU)."""

import ctypes

import numpy as np
import pytest

from invariant_vd_step_gb300 import build, vd


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    vd.lib()


def refused(code, f, *a, **k):
    with pytest.raises(vd.VDError) as e:
        f(*a, **k)
    assert e.value.code == code, e.value


def test_alloc_retain_release():
    p = vd.Pages(6)
    assert p.free == 6
    assert p.alloc(4).tolist() == [0, 1, 2, 3] and p.free == 2
    p.release([1])
    assert p.alloc(2).tolist() == [1, 4]
    p.retain([2, 2, 3])
    assert p.refs(2) == 3 and p.refs(3) == 2 and p.refs(5) == 0
    p.release([2, 2])
    assert p.refs(2) == 1 and p.free == 1
    refused(4, p.alloc, 2)
    assert p.free == 1
    refused(1, p.release, [3, 0, 2, 2])   # the last one no longer referenced: nothing changed
    assert [p.refs(i) for i in range(6)] == [1, 1, 1, 2, 1, 0] and p.free == 1
    refused(1, p.retain, [5])
    refused(3, p.retain, [6])
    refused(3, p.release, [-1])
    refused(1, p.release, [2 ** 40])
    p.retain([])
    p.release([])
    assert p.alloc(0).size == 0
    assert p.refs(6) == -1 and p.refs(-1) == -1


def test_fork_shares_complete_pages_and_copies_the_rest():
    p = vd.Pages(12)
    t = p.alloc(5)
    out, src, dst = p.fork(t, 4, 3)
    assert out.shape == (3, 5) and (out[:, :4] == t[:4]).all()
    assert sorted(out[:, 4].tolist()) == [5, 6, 7] and src.tolist() == [4] * 3 and dst.tolist() == out[:, 4].tolist()
    assert [p.refs(i) for i in range(8)] == [4, 4, 4, 4, 1, 1, 1, 1]
    for row in out:
        p.release(row)
    assert p.free == 7 and all(p.refs(i) == 1 for i in range(5))
    out, src, dst = p.fork(t, 5, 2)       # nothing is being filled
    assert src.size == 0 and (out == t).all() and p.refs(0) == 3
    out, src, dst = p.fork(t, 0, 1)       # nothing complete
    assert src.tolist() == t.tolist() and not set(dst) & set(t)
    refused(4, p.fork, t, 0, 1)           # 2 pages left
    assert p.free == 2 and p.refs(0) == 3
    refused(1, p.fork, t, 6, 1)
    refused(1, p.fork, [11], 0, 1)
    assert p.fork(t, 4, 0)[0].shape == (0, 5)
    assert p.fork([], 0, 3)[0].shape == (3, 0)


@pytest.mark.parametrize("seed", range(6))
def test_compaction_keeps_what_tables_say(seed):
    rng = np.random.default_rng(seed)
    N = int(rng.integers(1, 60))
    p = vd.Pages(N)
    p.alloc(N)
    content = np.arange(N) * 10           # what each page holds
    drop = rng.permutation(N)[:int(rng.integers(0, N + 1))]
    p.release(drop)
    live = np.setdiff1d(np.arange(N), drop)
    tables = np.full((3, 8), -1, np.int32)
    if len(live):
        tables[:2] = rng.choice(live, (2, 8))
        p.retain(tables[:2].reshape(-1))
    before = np.where(tables >= 0, content[np.maximum(tables, 0)], -1)
    refs = {int(content[i]): p.refs(i) for i in live}
    total, moves = 0, 1
    while moves:
        src, dst = p.compact(tables, max_moves=int(rng.integers(1, 5)))
        assert not set(src) & set(dst) and len(set(dst)) == len(dst)
        content[dst] = content[src]
        moves = len(src)
        total += moves
        assert (np.where(tables >= 0, content[np.maximum(tables, 0)], -1) == before).all()
    assert [p.refs(i) > 0 for i in range(N)] == [True] * len(live) + [False] * (N - len(live))
    assert p.free == N - len(live) and total == int((live >= len(live)).sum())
    assert {int(content[i]): p.refs(i) for i in range(len(live))} == refs


def test_compaction_refuses_tables_of_free_pages():
    p = vd.Pages(4)
    p.alloc(3)
    p.release([0])
    refused(1, p.compact, np.array([0], np.int32))
    refused(3, p.compact, np.array([4], np.int32))
    refused(1, p.compact, np.array([1], np.int64))
    refused(1, p.compact, np.array([1], np.int32), max_moves=-1)
    src, dst = p.compact(np.array([-1], np.int32))
    assert src.tolist() == [2] and dst.tolist() == [0]


def test_null_arguments():
    L = vd.lib()
    h = ctypes.c_void_p()
    assert L.vd_pages_create(0, ctypes.byref(h)) == 1 and L.vd_pages_create(4, None) == 1
    assert L.vd_pages_free(None) == -1 and L.vd_pages_refs(None, 0) == -1
    assert L.vd_pages_alloc(None, 1, None) == 1 and L.vd_pages_retain(None, 0, None) == 1
    assert L.vd_pages_compact(None, 0, None, None, None, 0, None) == 1
    assert L.vd_kv_copy_pages(None, 1, None, None, None) == 1 and L.vd_kv8_copy_pages(None, 1, None, None, None) == 1
    assert L.vd_kv8_create(None, 0, 1, None, 0, ctypes.byref(h)) == 1
    assert L.vd_kv8_plan_create(None, 1, ctypes.byref(h)) == 1
    assert L.vd_kv8_plan_make(None, None, None, None, None) == 1
    assert L.vd_op_kv8_attention(None, None, None, 0, None, None, None) == 1
    assert L.vd_step_kv8(None, None, None, None, None) == 1
    assert L.vd_kv8_seal(None, None, -1, 0, None, None, None) == 1
    assert L.vd_kv8_bytes(None, 4) == 0
    L.vd_destroy_kv8(None)
    L.vd_destroy_kv8_plan(None)
    L.vd_destroy_pages(None)
