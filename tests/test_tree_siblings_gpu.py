"""Drafted nodes whose V holds infinities or NaN: the rows that do not see them, and those that do, are the decoded
paths' rows bit for bit."""

import numpy as np
import pytest
import torch

from gpu_util import bits, ready
from tree_scenario import TreeScenario, make_tree, path_of, tree_spec

pytestmark = pytest.mark.gpu


def poison(sc, r, node, value, dims):
    """Sets V of a node of request r, in its slot and in every decoded path that holds it."""
    view, (c, parent) = sc.pool.view(), sc.trees[r]

    def put(table, slot):
        view[:, int(table[slot // 16]), 1, :, slot % 16, dims] = value
    put(sc.tables[r], c + node)
    for rr, i, _, table in sc.paths:
        if rr == r and node in path_of(parent, i):
            put(table, c + path_of(parent, i).index(node))


# trees enough for a warp to fold several nodes at once (more than 2 x 152 x 4 nodes x KV heads, half of it at head
# dim 256), of every shape, behind prefixes that end anywhere in a tile
@pytest.mark.parametrize("window", [0, 9, 40])
@pytest.mark.parametrize("Hq,Hkv,hd,B,n", [(8, 8, 64, 12, 16), (32, 8, 128, 10, 18), (16, 4, 256, 12, 15), (16, 8, 128, 9, 40)])
def test_siblings_of_nodes_that_are_not_finite(Hq, Hkv, hd, B, n, window):
    ready()
    kinds = ["random", "star", "comb", "chain"]
    trees = [([0, 1, 30, 31, 32, 45, 63, 500, 512, 77, 90, 1][r], make_tree(kinds[r % 4], n, r)) for r in range(B)]
    sc = TreeScenario(tree_spec(Hq, Hkv, hd, window), trees, seed=hd + n)
    finite = sc.attention()
    np.testing.assert_array_equal(bits(finite), bits(sc.decoded()))
    inf, nan = float("inf"), float("nan")
    sick = set()
    for r in range(B):
        for node, value, dims in [(n - 1, inf, slice(None)), (n // 2, nan, slice(3, 4)), (3, -inf, slice(hd - 5, hd)),
                                  (5, inf, slice(0, 2))][:1 + r % 4]:
            poison(sc, r, node, value, dims)
            sick.add((r, node))
    got, ref = sc.attention(), sc.decoded()
    np.testing.assert_array_equal(bits(got), bits(ref))
    # and rows that see no such node are what they were
    keep = [k for k, (r, i, _, _) in enumerate(sc.paths)
            if not any((r, j) in sick for j in path_of(sc.trees[r][1], i))]
    assert len(keep) > B and torch.isfinite(got[keep].float()).all() and not torch.isfinite(got.float()).all()
    np.testing.assert_array_equal(bits(got[keep]), bits(finite[keep]))
    assert sc.model.device_status() == 0


@pytest.mark.parametrize("window", [0, 9, 40])
@pytest.mark.parametrize("Hq,Hkv,hd,n", [(8, 2, 128, 210), (4, 2, 256, 110)])
def test_long_tails_with_nodes_that_are_not_finite(Hq, Hkv, hd, n, window):
    """Trees whose tails shared memory does not hold; also ancestors that a window hides within its lowest tile, whose
    weight is zero and whose values enter the decoded path's products all the same."""
    ready()
    trees = [(45, make_tree("chain", n)), (31, make_tree("comb", n)), (500, make_tree("random", 12, 1))]
    sc = TreeScenario(tree_spec(Hq, Hkv, hd, window), trees, seed=hd + window)
    for r, node, value in [(0, 60, float("inf")), (0, 101, float("nan")), (1, 80, float("-inf")), (1, 31, float("inf")),
                           (2, 4, float("nan"))]:
        poison(sc, r, node, value, slice(2, 9))
    got, ref = sc.attention(), sc.decoded()
    np.testing.assert_array_equal(bits(got), bits(ref))
    assert torch.isfinite(got.float()).any() and not torch.isfinite(got.float()).all()
    assert sc.model.device_status() == 0
