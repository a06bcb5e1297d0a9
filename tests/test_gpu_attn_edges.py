"""Calls of gdn_attn.h at the ends of what is allowed."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from attn_cases import (BF16, E4M3, HALF, Paged, ancestors, attend, bits_of, close, generator, i32, randn,  # noqa: E402
                        random_tree, tolerance)
from test_gpu_attn import TWO, causal, check_verify  # noqa: E402

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


def one_sequence(kind, p, H_q, seed=1):
    """A call of `kind` on p's only sequence: (queries, the mask of what they see, what makes the call, its weights)"""
    d, keys = p.k.shape[3], p.counts[0]
    n = {"decode": 1, "prefill": 100, "verify": 45}[kind]
    q = randn(generator(seed), n, H_q, d).to(BF16)
    if kind == "decode":
        return q, torch.ones(1, keys, dtype=torch.bool), lambda st=None: gdn.gdn_attn_decode(
            p.cache(), q, p.table, i32(keys), seq_status=st), TWO
    if kind == "prefill":
        return q, causal(n, keys), lambda st=None: gdn.gdn_attn_prefill(
            p.cache(), q, i32(0, n), p.table, i32(keys), seq_status=st), HALF
    tree = ancestors(random_tree(n, seed))[1]
    mask = torch.cat([torch.ones(n, keys - n, dtype=torch.bool), tree], 1)
    bits = bits_of(tree).cuda()[None]
    return q, mask, lambda st=None: gdn.gdn_attn_verify(p.cache(), q[None], bits, p.table, i32(keys - n), seq_status=st)[0], HALF


def spoil(p, pool, token, head, element, bad):
    x = p.get(pool, 0, torch.tensor([token]))
    x[:, head, element] = bad
    p.put(pool, 0, torch.tensor([token]), x)


@pytest.mark.parametrize("kind", ["prefill", "verify"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("size", [30.0, float("inf")])
def test_large_scores_of_other_rows_leave_no_trace(kind, d, page, size):
    """rows of a tile that do not see a key are the same to the last bit, however large its scores are for their neighbours"""
    H, group = 2, 3
    p = Paged([300], H, d, page)
    q, mask, run, _ = one_sequence(kind, p, H * group)
    clean = run()
    for token in (262, 285):
        spoil(p, p.k, token, slice(None), slice(None), size)
        sees = mask[:, token].cuda()
        got = run()
        assert sees.any() and (~sees).any()
        mine = ~(mask[:, 262].cuda() | sees)
        assert torch.equal(got[mine], clean[mine]) and not torch.equal(got, clean)


NOT_FINITE = [(BF16, float("nan")), (BF16, float("inf")), (BF16, float("-inf")), (E4M3, float("nan"))]


@pytest.mark.parametrize("kind", ["decode", "prefill", "verify"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("dtype,bad", NOT_FINITE)
@pytest.mark.parametrize("token", [20, 285])  # among what all queries see, and among what some see
def test_a_key_that_is_not_finite(kind, d, page, dtype, bad, token):
    """scores of NaN and +inf make a row NaN, one of -inf is a weight of zero, whoever does not see the key has no trace of it"""
    H, group, element = 2, 3, 5
    p = Paged([300], H, d, page, dtype)
    q, mask, run, weights = one_sequence(kind, p, H * group)
    clean = run()
    spoil(p, p.k, token, 1, element, bad)
    got = run()
    assert torch.equal(got[:, :group], clean[:, :group])
    sees = mask[:, token].cuda()
    assert torch.equal(got[~sees], clean[~sees]) and sees.any()
    score = q[:, group:, element].float() * bad
    gone = sees[:, None] & (score == -float("inf"))
    lost = sees[:, None] & ~gone
    assert got[:, group:][lost].isnan().all() and lost.any() and (gone.any() or bad != bad)
    if gone.any():
        without = mask.clone()
        without[:, token] = False
        ref = attend(q, p.real["k"][0], p.real["v"][0], without.cuda(), d ** -0.5)
        tol = tolerance(*ref, d, weights)
        close(got[:, group:][gone], ref[0][:, group:][gone], tol[:, group:][gone])


@pytest.mark.parametrize("kind", ["decode", "prefill", "verify"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [8, 16])
@pytest.mark.parametrize("dtype,bad", NOT_FINITE)
@pytest.mark.parametrize("token", [20, 285])
def test_a_value_that_is_not_finite(kind, d, page, dtype, bad, token):
    """makes that element of who sees it infinite or NaN, and nothing else"""
    H, group, element = 2, 3, 5
    p = Paged([300], H, d, page, dtype)
    q, mask, run, _ = one_sequence(kind, p, H * group)
    clean = run()
    spoil(p, p.v, token, 1, element, bad)
    got = run()
    sees = mask[:, token].cuda()
    hit = got[sees][:, group:, element]
    assert not hit.isfinite().any() and hit.numel()
    if bad != bad:
        assert hit.isnan().all()
    got[sees.nonzero(), torch.arange(group, 2 * group, device="cuda"), element] = clean[
        sees.nonzero(), torch.arange(group, 2 * group, device="cuda"), element]
    assert torch.equal(got, clean)


def test_only_keys_with_scores_of_minus_infinity():
    """weights of zero: as if nothing were visible"""
    p = Paged([3], 1, 64)
    q = torch.ones(1, 2, 64, dtype=BF16, device="cuda")
    for t in range(3):
        spoil(p, p.k, t, 0, 7, -float("inf"))
    assert (gdn.gdn_attn_decode(p.cache(), q, p.table, i32(3)) == 0).all()
    assert (gdn.gdn_attn_prefill(p.cache(), q, i32(0, 1), p.table, i32(3)) == 0).all()


@pytest.mark.parametrize("kind", ["decode", "prefill", "verify"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("page", [1, 8, 16, 64])
def test_pages_outside_the_pool(kind, d, dtype, page):
    """keys there are left out: among those before a tree, in it, and the last"""
    H, group, keys = 2, 3, 330
    p = Paged([keys], H, d, page, dtype)
    q, mask, run, weights = one_sequence(kind, p, H * group)
    gone = sorted({t // page for t in (3, 140, 141, 290, 300, keys - 1)})
    for i, g in enumerate(gone):
        p.table[0, g] = (-1, p.k.shape[0], 2 ** 31 - 1, -2 ** 31)[i % 4]
    mask[:, [t for t in range(keys) if t // page in gone]] = False
    st = i32(9)
    got = run(st)
    ref = attend(q, p.real["k"][0], p.real["v"][0], mask.cuda(), d ** -0.5)
    close(got, ref[0], tolerance(*ref, d, weights))
    assert st.tolist() == [2]


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_commit_of_layers_that_share_a_cache(dtype):
    """the path moves once, also where the cache is in two launches of the call, or keys alone are shared"""
    N, lengths = 60, [30, 7]
    anc = torch.zeros(2, N, 2, dtype=torch.int32)
    anc[:, N - 1] = bits_of(torch.arange(N).expand(N, N) % 3 == 2)[0]  # nodes 2, 5, 8, ... 59
    anc = anc.cuda()
    accepted, length = i32(N - 1, N - 1), i32(*lengths)
    ps = [Paged([n + N for n in lengths], 2, 64, dtype=dtype, seed=s) for s in (1, 1, 2, 2)]
    single, shared = ps[0::2], ps[1::2]
    for p in ps[1:]:
        p.table.copy_(ps[0].table)
    for a, b in zip(single, shared):
        for x in "kv":
            getattr(b, x).view(torch.uint8).copy_(getattr(a, x).view(torch.uint8))
    gdn.gdn_kv_commit([p.cache() for p in single], anc, accepted, single[0].table, length)
    first, second = (p.cache() for p in shared)
    keys_only = gdn.GdnKvCache(shared[0].k, shared[1].v, shared[0].k_scale, shared[0].v_scale)
    many = [first] * 3 + [keys_only] + [second] * 40 + [first, keys_only]
    new = gdn.gdn_kv_commit(many, anc, accepted, shared[0].table, length)
    assert new.tolist() == [n + N // 3 for n in lengths]
    for a, b in zip(single, shared):
        for x in "kv":
            assert torch.equal(getattr(a, x).view(torch.uint8), getattr(b, x).view(torch.uint8))
