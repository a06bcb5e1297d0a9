"""gdn_linear over sizes that its other tests leave out.  Tolerances as there."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from test_gpu_layer import BF16, F32, LINEAR_TOL, check, gpu, say  # noqa: E402,F401
from test_layer_linear_choice import SHAPES, choice  # noqa: E402

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


def rows_of(n, K, stride, scale, gen):
    """[n][K] rows `stride` apart with NaN between them."""
    wide = torch.full((n, stride), float("nan"), dtype=BF16, device="cuda")
    wide[:, :K] = torch.randn(n, K, generator=gen, device="cuda") * scale
    return wide[:, :K]


@pytest.mark.parametrize("M,N,K,stride,kernel,tail,cut", SHAPES)
def test_every_kernel(M, N, K, stride, kernel, tail, cut):
    say(f"[linear] {M} x {N} x {K}, rows {stride or K} apart: kernel {kernel}, tail {tail}, cut {cut}")
    assert choice(M, N, K, stride) == (kernel, tail, cut)
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    x, w = rows_of(M, K, stride or K, 1.0, gen), rows_of(N, K, stride or K, K ** -0.5, gen)
    y = gdn.gdn_linear(x, w, y_dtype=F32)
    want = x.double().contiguous() @ w.double().t().contiguous()
    check(y, want, LINEAR_TOL, "y")
    bias, res = torch.randn(N, generator=gen, device="cuda"), torch.randn(M, N, generator=gen, device="cuda").to(BF16)
    y2 = gdn.gdn_linear(x, w, bias=bias, act="silu", residual=res, scale=0.7)
    z = want + bias.double()
    check(y2, res.double() + 0.7 * z * torch.sigmoid(z), LINEAR_TOL, "with bias, silu and residual")
    x[M // 2, K - 1] = float("inf")  # the last element of a row: that row alone
    y3 = gdn.gdn_linear(x, w, y_dtype=F32)
    assert torch.isinf(y3[M // 2]).all()
    assert torch.equal(y3[:M // 2], y[:M // 2]) and torch.equal(y3[M // 2 + 1:], y[M // 2 + 1:])
