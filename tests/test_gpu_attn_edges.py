"""Calls of gdn_attn.h at the ends of what is allowed."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from attn_cases import BF16, Paged, ancestors, i32, random_tree  # noqa: E402
from test_gpu_attn import check_verify  # noqa: E402

pytestmark = pytest.mark.gpu


def test_trees_without_nodes():
    """an output of no rows, and a verdict on each prefix"""
    p = Paged([5, 40, 7], 2, 64)
    p.table[1, 2] = -1
    q = torch.empty(3, 0, 4, 64, dtype=BF16, device="cuda")
    anc = torch.empty(3, 0, 1, dtype=torch.int32, device="cuda")
    st = i32(9, 9, 9)
    for gate in (None, q):
        o = gdn.gdn_attn_verify(p.cache(), q, anc, p.table, i32(5, 40, 99), gate=gate, seq_status=st)
        assert o.shape == q.shape and st.tolist() == [0, 2, 2]
    length = i32(5, 32, 7)
    assert gdn.gdn_kv_commit(p.cache(), anc, i32(-1, -1, -1), p.table, length, seq_status=st).tolist() == [5, 32, 7]
    assert st.tolist() == [0, 0, 0]


@pytest.mark.parametrize("d,group", [(128, 4), (64, 4), (256, 8)])
def test_a_workspace_for_the_largest_tree_serves_smaller_ones(d, group):
    """teams are whole, so some smaller trees ask for more"""
    most, H, prefix = 160, 2, [3000, 5, 900]
    p = Paged([n + most for n in prefix], H, d)

    def need(N):
        return gdn.gdn_attn_workspace_bytes("verify", p.cache(), len(prefix), N, H * group, p.table.shape[1])

    nbytes = need(most)
    ws = torch.full((nbytes + 4096,), 93, dtype=torch.uint8, device="cuda")
    sizes = [most, 128, 96, 33, 7, 1]
    assert any(need(N) > nbytes for N in sizes)
    for N in sizes:
        masks = [ancestors(random_tree(N, N + b))[1] for b in range(len(prefix))]
        check_verify(p, prefix, masks, H * group, N, workspace=ws[:nbytes])
        assert (ws[nbytes:] == 93).all()
