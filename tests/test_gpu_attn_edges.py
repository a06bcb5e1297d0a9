"""Calls of gdn_attn.h at the ends of what is allowed."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from attn_cases import BF16, Paged, i32  # noqa: E402

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
