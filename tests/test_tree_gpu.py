"""The ancestors of a tree of drafted tokens and the walk that accepts a path, against
plain forms."""
import numpy as np
import pytest
import torch

import sparse_head_attention_gb300 as ea
from gpu_helpers import check_no_device_error, gpu_device
from tree_reference import accept, plan, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    return gpu_device()


def _i32(v, dev):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)


@pytest.mark.parametrize("kind", ["tree", "chain", "star", "forest"])
@pytest.mark.parametrize("B,T", [(1, 1), (2, 2), (4, 31), (3, 33), (5, 64), (3, 100), (2, 128)])
def test_plan_and_accept(dev, kind, B, T):
    p = random_tree(B, T, 7 * T + B, kind)
    n = [T, 1, 0, T // 2, T - 1][:B]
    ws = ea.cache_workspace(dev)
    depth, mask = ea.ea_tree_plan(_i32(p, dev), _i32(n, dev), workspace=ws)
    d, m = plan(p, n)
    assert np.array_equal(depth.cpu().numpy(), d) and np.array_equal(mask.cpu().numpy(), m)
    r = np.random.RandomState(T)
    for vocab in (1, 2, 5):
        tok, tgt = r.randint(0, vocab, (B, T)), r.randint(0, vocab, (B, T))
        tgt[:, ::5] = -1                                 # a target no token equals
        got = ea.ea_tree_accept(_i32(tok, dev), _i32(p, dev), _i32(tgt, dev), _i32(n, dev), workspace=ws)
        for a, b in zip(got, accept(tok, p, tgt, n)):
            assert np.array_equal(a.cpu().numpy(), b)
    check_no_device_error(ws)
    full, whole = ea.ea_tree_plan(_i32(p, dev))          # n_nodes left out
    d, m = plan(p, [T] * B)
    assert np.array_equal(full.cpu().numpy(), d) and np.array_equal(whole.cpu().numpy(), m)


def test_bad_parents_and_counts(dev):
    p = np.array([[-1, 0, 2, 1], [-2, 0, 1, 2], [-1, 5, 1, 0], [-1, 0, 1, 2]], np.int32)
    n = [4, 4, 4, 5]
    fixed = np.array([[-1, 0, -1, 1], [-1, 0, 1, 2], [-1, -1, 1, 0], [-1] * 4], np.int32)
    ws = ea.cache_workspace(dev)
    depth, mask = ea.ea_tree_plan(_i32(p, dev), _i32(n, dev), workspace=ws)
    assert ea.ea_check_errors(ws) == 6
    d, m = plan(fixed, [4, 4, 4, 0])
    assert np.array_equal(depth.cpu().numpy(), d) and np.array_equal(mask.cpu().numpy(), m)
    z = np.zeros((4, 4), np.int32)
    got = ea.ea_tree_accept(_i32(z, dev), _i32(p, dev), _i32(z, dev), _i32(n, dev), workspace=ws)
    assert ea.ea_check_errors(ws) == 6
    for a, b in zip(got, accept(z, fixed, z, [4, 4, 4, 0])):
        assert np.array_equal(a.cpu().numpy(), b)
    # what lies behind a sequence's nodes is not looked at
    ea.ea_tree_plan(_i32([[-1, 0, 9, -7]], dev), _i32([2], dev), workspace=ws)
    check_no_device_error(ws)
