"""gdn_linear over sizes that its other tests leave out.  Tolerances as there."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from test_gpu_layer import BF16, F32, LINEAR_TOL, check, gpu, say  # noqa: E402,F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,K", [((1 << 28) + 5, 1), ((1 << 30) + 3, 8), ((1 << 31) - 1, 8)])
def test_more_workgroups_than_one_grid_dimension_holds(M, K):
    """2^22 tiles of 1024 threads (rows of no alignment), 2^24 of 256, and a row count at the end of int32"""
    say(f"[linear] {M} x 1 x {K}")
    w = torch.full((1, K), 0.5, dtype=BF16, device="cuda")
    if K == 1:
        x = (torch.arange(M, device="cuda", dtype=torch.int32) % 251).to(BF16)[:, None]
    else:
        x = torch.ones(1, K, dtype=BF16, device="cuda").expand(M, K)
    y = torch.full((M, 1), -1.0, dtype=BF16, device="cuda")
    gdn.gdn_linear(x, w, y=y)
    for at in range(0, M, 1 << 27):  # multiples of a half below 128: exact
        want = 0.5 * x[at:at + (1 << 27)].sum(1, keepdim=True)
        assert torch.equal(y[at:at + (1 << 27)], want)
