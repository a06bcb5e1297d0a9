"""The example's blocks give the same outputs and states along their three
paths: packed prompts, single tokens and a verified tree.

The paths share weights and inputs and differ in where fp32 is rounded to
bf16 (half a step of 2^-8).  A row passes about five such roundings per block
(norm, projection, normalised q and k, gate, projection), so two blocks differ
by some sqrt(10) 2^-9 = 6e-3 at most of them; three times that is allowed.
States come before the last gate and projection and get the same bound.
"""
import importlib.util
import os

import pytest

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_loop.py")
BOUND = 2e-2


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    {},
    dict(lengths=(5, 8, 64, 1), D=200, H_k=1, H_v=1, d=64, nodes=7, seed=3),
    dict(lengths=(400,), D=512, H_k=4, H_v=8, d=128, nodes=130, tokens=1, seed=5),
])
def test_example_paths_agree(kw):
    spec = importlib.util.spec_from_file_location("decode_loop", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    far = example.main(**kw)
    print(far)
    for name, value in far.items():
        assert value <= BOUND, (name, value)
