"""What the Python binding of gdn_layer.h checks and allocates."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from test_gpu_layer import BF16, F32, gpu, i32, make  # noqa: E402,F401

pytestmark = pytest.mark.gpu

WORKSPACES = [  # none of these is memory that a kernel may write to
    (lambda n: torch.empty(n, dtype=torch.uint8), ValueError),
    (lambda n: torch.empty(1, dtype=torch.uint8, device="cuda").expand(n), ValueError),
    (lambda n: torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2], ValueError),
    (lambda n: torch.empty(n, device="cuda"), TypeError),
    (lambda n: bytearray(n), TypeError),
]


@pytest.mark.parametrize("make_ws,error", WORKSPACES)
def test_a_workspace_is_checked(make_ws, error):
    d = make(200)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    cu = i32(0, 200)
    need = gdn.gdn_prefill_workspace_bytes(d["q"], d["v"], cu)
    assert need > 0
    with pytest.raises(error, match="workspace"):
        gdn.gdn_prefill(*args, cu, d["S"], workspace=make_ws(need))
    x, w = (torch.zeros(600, 129, dtype=BF16, device="cuda")[:, :128] for _ in range(2))  # rows that are copied first
    with pytest.raises(error, match="workspace"):
        gdn.gdn_linear(x, w, workspace=make_ws(1 << 20))
    y = gdn.gdn_linear(x, w, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert (y == 0).all()
