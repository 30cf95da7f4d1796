"""The example that runs the tree verification calls together."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import gated_delta_rule_05_gb300 as m
    m.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "examples", "tree_verify.py")
    spec = importlib.util.spec_from_file_location("tree_verify", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("d", [32, 64])
def test_trees_give_the_tokens_of_one_at_a_time(example, d):
    out, plain, steps = example.main(["--new-tokens", "40", "--d", str(d)])
    assert out == plain and all(len(x) == 40 for x in out)
    assert steps < 40, "no drafted token was ever accepted"


def test_bf16(example):
    out, _, steps = example.main(["--new-tokens", "24", "--d", "128", "--dtype", "bf16",
                                  "--sequences", "3", "--nodes", "20"])
    assert all(len(x) == 24 for x in out) and steps < 24
