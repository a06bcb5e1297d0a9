"""The attention of gdn_attn.h where sequences, tiles or callers are many."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from attn_cases import BF16, E4M3, Paged, ancestors, attend, bits_of, close, generator, i32, randn, random_tree, tolerance  # noqa: E402
from test_gpu_attn import TWO, check_decode, check_prefill, check_verify  # noqa: E402

pytestmark = pytest.mark.gpu


def mixed(n, most, seed, long=()):
    """n lengths below `most`, some of them zero, and at the places of `long` the lengths there"""
    x = torch.randint(0, most, (n,), generator=torch.Generator().manual_seed(seed)).tolist()
    for at, length in dict(long).items():
        x[at] = length
    return x


@pytest.mark.parametrize("d,H,group,dtype", [(128, 1, 2, BF16), (64, 2, 1, E4M3), (256, 1, 17, BF16)])
def test_decode_of_more_sequences_than_workgroups(d, H, group, dtype):
    """the parts of the long ones are joined, whose neighbours are whole"""
    lengths = mixed(1100, 40, 5, {0: 900, 63: 4000, 64: 1, 500: 2500, 501: 1300, 1099: 5000})
    p = Paged(lengths, H, d, 16, dtype, seed=d)
    print(check_decode(p, lengths, H * group)[1])


@pytest.mark.parametrize("d,H,group,dtype", [(128, 2, 4, BF16), (64, 1, 3, E4M3), (256, 1, 8, BF16)])
def test_prefill_of_many_prompts(d, H, group, dtype):
    new = mixed(150, 30, 6, {2: 0, 63: 700, 64: 257, 149: 300})
    lengths = [n + more for n, more in zip(new, mixed(150, 200, 7, {64: 3000, 100: 2000}))]
    p = Paged(lengths, H, d, 32, dtype, seed=d)
    print(check_prefill(p, new, lengths, H * group)[1])


@pytest.mark.parametrize("d,H,group,N,dtype", [(128, 1, 4, 9, BF16), (128, 2, 8, 64, BF16), (64, 2, 6, 33, E4M3),
                                               (256, 2, 8, 64, BF16)])
def test_verify_of_many_trees(d, H, group, N, dtype):
    """fewer and more tiles than teams of workgroups"""
    prefix = mixed(140, 150, 8, {0: 3000, 63: 0, 64: 2000, 139: 1500})
    p = Paged([n + N for n in prefix], H, d, 16, dtype, seed=N)
    masks = [ancestors(random_tree(N, b))[1] for b in range(len(prefix))]
    print(check_verify(p, prefix, masks, H * group, N)[1])


@pytest.mark.parametrize("d,group", [(256, 130), (64, 260)])
def test_verify_of_more_tiles_than_workgroups(d, group):
    """one team, whose keys are not divided: no workspace"""
    N, prefix = 256, [0, 90]
    p = Paged([n + N for n in prefix], 1, d, 16)
    assert gdn.gdn_attn_workspace_bytes("verify", p.cache(), 2, N, group, p.table.shape[1]) == 0
    masks = [ancestors(random_tree(N, b))[1] for b in range(2)]
    print(check_verify(p, prefix, masks, group, N)[1])


def test_sequences_that_share_pages():
    """a prefix in common, the same row of the table twice"""
    p = Paged([700], 2, 128, 16)
    lengths = [700, 333, 700, 16, 0, 1]
    q = randn(generator(3), len(lengths), 8, 128).to(BF16)
    got = gdn.gdn_attn_decode(p.cache(), q, p.table.expand(len(lengths), -1), i32(*lengths))
    for b, n in enumerate(lengths):
        k, v = (p.real[x][0][:n] for x in ("k", "v"))
        ref = attend(q[b:b + 1], k, v, torch.ones(1, n, dtype=torch.bool, device="cuda"), 128 ** -0.5)
        close(got[b:b + 1], ref[0], tolerance(*ref, 128, TWO), f"sequence {b}")


@pytest.mark.parametrize("d", [128, 256])
def test_two_graphs_with_one_workspace(d):
    """replayed in turn, with eager calls between them"""
    lengths, N = [2000, 3, 900], 20
    p = Paged([n + N for n in lengths], 2, d)
    cache, length = p.cache(), i32(*lengths)
    gen = generator(1)
    q, tree_q = randn(gen, 3, 8, d).to(BF16), randn(gen, 3, N, 8, d).to(BF16)
    bits = torch.stack([ancestors(random_tree(N, b))[0] for b in range(3)]).cuda()
    need = max(gdn.gdn_attn_workspace_bytes(kind, cache, 3, n, 8, p.table.shape[1])
               for kind, n in (("decode", 3), ("verify", N), ("prefill", 3 * N)))
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    flat = tree_q.flatten(0, 1)
    calls = [lambda o=None: gdn.gdn_attn_decode(cache, q, p.table, length, o=o, workspace=ws),
             lambda o=None: gdn.gdn_attn_verify(cache, tree_q, bits, p.table, length, o=o, workspace=ws),
             lambda o=None: gdn.gdn_attn_prefill(cache, flat, i32_cu, p.table, more, o=o, workspace=ws)]
    i32_cu, more = i32(0, N, 2 * N, 3 * N), length + N
    want = [f() for f in calls]
    out = [torch.empty_like(x) for x in want]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for f, o in zip(calls, out):
            f(o)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for f, o in zip(calls, out):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            f(o)
    for i in range(6):
        for x in out:
            x.zero_()
        for at in ((0, 1, 2), (2, 0, 1), (1, 1, 0, 2))[i % 3]:
            graphs[at].replay()
            if i > 2:
                assert torch.equal(calls[(at + 1) % 3](), want[(at + 1) % 3])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    """calls that overlap have workspaces of their own"""
    p = Paged([9000, 500, 33], 2, 128)
    cache, length = p.cache(), i32(9000, 500, 33)
    q = [randn(generator(s), 3, 8, 128).to(BF16) for s in range(2)]
    want = [gdn.gdn_attn_decode(cache, x, p.table, length) for x in q]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[gdn.gdn_attn_decode(cache, x, p.table, length, stream=s) for _ in range(8)] for x, s in zip(q, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(y, w) for x, w in zip(got, want) for y in x)


def test_one_page_row_or_head_has_no_stride():
    """what a view has there is any number"""
    gen = generator(2)
    page = randn(gen, 16, 64).to(BF16)
    q, table = randn(gen, 1, 2, 64).to(BF16), i32(0).view(1, 1)
    plain = gdn.GdnKvCache(page.view(1, 16, 1, 64), page.view(1, 16, 1, 64))
    odd = page.as_strided((1, 16, 1, 64), (7, 64, 3, 1))
    cache = gdn.GdnKvCache(odd, odd)
    want = gdn.gdn_attn_decode(plain, q, table, i32(11))
    assert torch.equal(gdn.gdn_attn_decode(cache, q, table, i32(11)), want)
    row = page[:5, :].as_strided((5, 1, 1, 64), (64, 1, 5, 1))  # pages of one token
    got = gdn.gdn_attn_decode(gdn.GdnKvCache(row, row), q, i32(0, 1, 2, 3, 4).view(1, 5), i32(5))
    assert torch.equal(got, gdn.gdn_attn_decode(plain, q, table, i32(5)))
