"""The example of tree decoding: the cache, its attention, the verify step and the commit together."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("tree_decoding", os.path.join(ROOT, "examples", "tree_decoding.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_tree_is_one():
    e = example()
    assert len(e.PARENTS) == len(e.CHOICE) and e.PARENTS[0] == -1
    assert all(0 <= p < i for i, p in enumerate(e.PARENTS) if i)
    siblings = list(zip(e.PARENTS[1:], e.CHOICE[1:]))
    assert len(set(siblings)) == len(siblings)


@pytest.mark.gpu
@pytest.mark.parametrize("batch, seed", [(1, 0), (5, 1)])
def test_trees_give_the_tokens_of_plain_decoding_in_fewer_passes(batch, seed):
    e = example()
    want = e.plain(batch, 40, seed)
    got, passes = e.with_trees(batch, 40, seed)
    assert got.tolist() == want.tolist()
    assert passes < 39
