"""The example's model verifies and commits trees of one size after another."""
import importlib.util

import pytest

torch = pytest.importorskip("torch")

from test_gpu_example import PATH  # noqa: E402


@pytest.mark.gpu
def test_trees_of_several_sizes():
    spec = importlib.util.spec_from_file_location("decode_loop", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model, same = (example.Model(2, 128, 1, 2, 64, seed=1) for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(2)
    for n in (5, 9, 5):
        x = torch.randn(2, n, 128, generator=gen, device="cuda").bfloat16()
        parent = torch.arange(-1, n - 1, dtype=torch.int32, device="cuda").repeat(2, 1)
        out = model.tree(x, parent)
        model.commit(torch.full((2,), n - 1, dtype=torch.int32, device="cuda"))
        one = torch.stack([same.token(x[:, t]) for t in range(n)], dim=1)
        assert example.rel(one, out) <= 2e-2  # as in the test of the example's paths
        for a, b in zip(model.states, same.states):
            assert example.rel(a, b) <= 2e-2
