"""The attention of gdn_attn.h against softmax attention in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from attn_cases import (BF16, E4M3, HALF, Paged, ancestors, attend, bits_of, close, generator, i32, randn,  # noqa: E402
                        random_tree, tolerance)

pytestmark = pytest.mark.gpu

TWO = HALF * HALF  # weights as two bf16


def gate_of(gen, shape, on):
    """A gate as a slice of wider rows."""
    return randn(gen, *shape[:-1], 2 * shape[-1]).to(BF16)[..., shape[-1]:] if on else None


def check_decode(p, lengths, H_q, seed=1, gate=False, scale=None, q_pad=0, status=None, **kw):
    H, d = p.k.shape[2:]
    gen = generator(seed)
    q = (2.0 * randn(gen, len(lengths), H_q * d + q_pad)).to(BF16)[:, :H_q * d].unflatten(1, (H_q, d))
    z = gate_of(gen, q.shape, gate)
    st = torch.full((len(lengths),), -7, dtype=torch.int32, device="cuda")
    got = gdn.gdn_attn_decode(p.cache(), q, p.table, i32(*lengths), gate=z, scale=scale, seq_status=st, **kw)
    worst = 0.0
    for b, n in enumerate(lengths):
        n = max(min(n, p.counts[b]), 0)
        k, v = (p.real[x][b][:n] for x in ("k", "v"))
        mask = torch.ones(1, n, dtype=torch.bool, device="cuda")
        ref = attend(q[b:b + 1], k, v, mask, d ** -0.5 if scale is None else scale, None if z is None else z[b:b + 1])
        worst = max(worst, close(got[b:b + 1], ref[0], tolerance(*ref, d, TWO), f"sequence {b} of {n}"))
    assert st.tolist() == (status or [0] * len(lengths))
    return got, worst


LENGTHS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130, 255, 256, 257, 700, 1025]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("H,group,page,layout", [(2, 8, 16, "rows"), (1, 1, 64, "heads"), (3, 7, 8, "both"),
                                                 (2, 16, 128, "wide"), (1, 17, 1, "rows"), (1, 40, 32, "heads")])
def test_decode_lengths_and_heads(d, dtype, H, group, page, layout):
    p = Paged(LENGTHS, H, d, page, dtype, seed=d + group, layout=layout)
    print(check_decode(p, LENGTHS, H * group, gate=group % 2 == 1, q_pad=8 * (group % 3))[1])


@pytest.mark.parametrize("d,H,group,dtype", [(128, 1, 4, BF16), (64, 2, 3, E4M3), (256, 1, 8, BF16), (128, 8, 4, E4M3)])
@pytest.mark.parametrize("lengths", [[40001], [1, 9000, 0, 17, 300], [3] * 70 + [20000] + [2] * 70])
def test_decode_long_and_uneven(d, H, group, dtype, lengths):
    p = Paged(lengths, H, d, 64, dtype, seed=3)
    print(check_decode(p, lengths, H * group, gate=True)[1])


def test_decode_shorter_than_the_cache():
    """rows behind a length are not seen, whatever they hold"""
    p = Paged([500, 300, 64, 1], 2, 128, 16)
    for n in ([499, 299, 63, 1], [257, 1, 32, 0]):  # never longer: what was overwritten stays behind
        for b, m in enumerate(n):
            rest = torch.arange(m, p.counts[b])
            p.put(p.k, b, rest, torch.full((len(rest), 2, 128), float("inf"), device="cuda").to(BF16))
            p.put(p.v, b, rest, torch.full((len(rest), 2, 128), float("nan"), device="cuda").to(BF16))
        check_decode(p, n, 8)


@pytest.mark.parametrize("scale", [0.0, 1e-3, 0.5, 3.0])
def test_decode_scales(scale):
    """a large scale leaves one weight of 1, a scale of zero the mean"""
    p = Paged([333, 1000, 5], 2, 64, 16)
    check_decode(p, [333, 1000, 5], 4, scale=scale)


def test_decode_bad_pages_and_lengths():
    """keys on pages outside the pool are left out; lengths are cut to the table"""
    p = Paged([100, 200, 300, 64], 2, 128, 16)
    p.table[0, 2], p.table[1, 0], p.table[1, 12] = -5, p.k.shape[0], 2 ** 31 - 1
    keep = [[t for t in range(n) if (b, t // 16) not in ((0, 2), (1, 0), (1, 12))] for b, n in enumerate(p.counts)]
    for b in range(2):
        for x in ("k", "v"):
            p.real[x][b] = p.real[x][b][keep[b]]
    p.counts = [len(x) for x in keep]
    gen = generator(4)
    q = randn(gen, 4, 8, 128).to(BF16)
    st = i32(9, 9, 9, 9)
    got = gdn.gdn_attn_decode(p.cache(), q, p.table, i32(100, 200, -3, 64), seq_status=st)
    assert st.tolist() == [2, 2, 2, 0] and (got[2] == 0).all()
    for b in (0, 1, 3):
        ref = attend(q[b:b + 1], p.real["k"][b], p.real["v"][b],
                     torch.ones(1, p.counts[b], dtype=torch.bool, device="cuda"), 128 ** -0.5)
        close(got[b:b + 1], ref[0], tolerance(*ref, 128, TWO))
    small = Paged([64], 1, 64, 16)
    st = i32(9)
    got = gdn.gdn_attn_decode(small.cache(), randn(gen, 1, 1, 64).to(BF16), small.table, i32(10 ** 9), seq_status=st)
    assert st.tolist() == [2] and not got.isnan().any()


def check_tiles(p, rows, prefix, H_q, masks, run, seed, gate, scale=None, weights=HALF):
    """`rows[b]` queries of sequence b over its first prefix + rows tokens under masks[b]; `run` makes the call."""
    H, d = p.k.shape[2:]
    gen = generator(seed)
    n = sum(rows)
    q = (2.0 * randn(gen, n, H_q * d + 8)).to(BF16)[:, :H_q * d].unflatten(1, (H_q, d))
    z = gate_of(gen, q.shape, gate)
    got = run(q, z)
    worst, at = 0.0, 0
    for b, m in enumerate(rows):
        keys = masks[b].shape[1]
        ref = attend(q[at:at + m], p.real["k"][b][:keys], p.real["v"][b][:keys], masks[b].cuda(),
                     d ** -0.5 if scale is None else scale, None if z is None else z[at:at + m])
        worst = max(worst, close(got[at:at + m], ref[0], tolerance(*ref, d, weights), f"sequence {b}"))
        at += m
    return got, worst


def causal(n, length):
    return torch.arange(length) <= torch.arange(length - n, length)[:, None]


def check_prefill(p, new, lengths, H_q, seed=1, gate=False, scale=None):
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st = torch.full((len(new),), -7, dtype=torch.int32, device="cuda")

    def run(q, z):
        return gdn.gdn_attn_prefill(p.cache(), q, i32(*cu), p.table, i32(*lengths), gate=z, scale=scale, seq_status=st)

    masks = [causal(n, m) for n, m in zip(new, lengths)]
    out = check_tiles(p, new, None, H_q, masks, run, seed, gate, scale)
    assert st.tolist() == [0] * len(new)
    return out


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("H,group,page,layout", [(2, 8, 16, "rows"), (1, 1, 64, "heads"), (2, 7, 8, "both"),
                                                 (1, 3, 1, "wide"), (1, 130, 32, "rows")])
def test_prefill_lengths_and_heads(d, dtype, H, group, page, layout):
    new = [0, 1, 3, 17, 64, 0, 129, 40, 1, 5]
    lengths = [7, 1, 3, 80, 64, 0, 129, 600, 513, 5]
    p = Paged(lengths, H, d, page, dtype, seed=d + group, layout=layout)
    print(check_prefill(p, new, lengths, H * group, gate=group % 2 == 1)[1])


@pytest.mark.parametrize("d,H,group,dtype", [(128, 1, 4, BF16), (64, 2, 3, E4M3), (256, 1, 8, BF16)])
def test_prefill_of_a_long_prompt(d, H, group, dtype):
    p = Paged([2500], H, d, 64, dtype)
    print(check_prefill(p, [2500], [2500], H * group)[1])


@pytest.mark.parametrize("d,H,group,dtype", [(128, 2, 4, BF16), (64, 1, 8, E4M3), (256, 1, 8, BF16)])
def test_prefill_of_few_tokens_behind_many(d, H, group, dtype):
    """the keys of a tile are divided, and its causal end lies in the middle of a part"""
    lengths, new = [9001, 300, 4100, 2], [37, 300, 1, 2]
    p = Paged(lengths, H, d, 32, dtype)
    print(check_prefill(p, new, lengths, H * group, gate=True)[1])


def check_verify(p, prefix, masks, H_q, N, seed=1, gate=False, scale=None, dev_bits=None, **kw):
    B = len(prefix)
    bits = torch.stack([bits_of(m) for m in masks]).cuda() if dev_bits is None else dev_bits
    whole = [torch.cat([torch.ones(N, n, dtype=torch.bool), m], 1) for n, m in zip(prefix, masks)]
    st = torch.full((B,), -7, dtype=torch.int32, device="cuda")

    def run(q, z):
        return gdn.gdn_attn_verify(p.cache(), q.unflatten(0, (B, N)), bits, p.table, i32(*prefix), scale=scale,
                                   gate=None if z is None else z.unflatten(0, (B, N)), seq_status=st, **kw).flatten(0, 1)

    out = check_tiles(p, [N] * B, None, H_q, whole, run, seed, gate, scale)
    assert st.tolist() == [0] * B
    return out


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("N,H,group,page", [(1, 2, 4, 16), (7, 1, 1, 8), (32, 2, 8, 16), (33, 1, 6, 64), (128, 1, 4, 16),
                                            (200, 1, 2, 128), (256, 1, 1, 1)])
def test_verify_trees(d, dtype, N, H, group, page):
    prefix = [0, 1, 63, 64, 65, 100, 700]
    p = Paged([n + N for n in prefix], H, d, page, dtype, seed=N, layout=["rows", "heads", "both", "wide"][N % 4])
    masks = [ancestors(random_tree(N, 10 * N + b))[1] for b in range(len(prefix))]
    print(check_verify(p, prefix, masks, H * group, N, gate=N % 2 == 1)[1])


@pytest.mark.parametrize("d,H,group,dtype", [(128, 2, 4, BF16), (64, 1, 8, E4M3), (256, 2, 8, BF16)])
def test_verify_behind_a_long_prefix(d, H, group, dtype):
    prefix, N = [20011, 3, 5000], 37
    p = Paged([n + N for n in prefix], H, d, 16, dtype)
    masks = [ancestors(random_tree(N, b))[1] for b in range(3)]
    print(check_verify(p, prefix, masks, H * group, N, gate=True)[1])


def test_verify_takes_what_tree_ancestors_writes():
    N = 70
    parent = [random_tree(N, s) for s in range(3)]
    anc, _, status = gdn.gdn_tree_ancestors(torch.tensor(parent, dtype=torch.int32, device="cuda"))
    assert status.tolist() == [0, 0, 0]
    p = Paged([50 + N, N, 333 + N], 2, 128)
    check_verify(p, [50, 0, 333], [ancestors(x)[1] for x in parent], 8, N, dev_bits=anc)


def test_rows_that_see_nothing_are_zero():
    N = 40
    mask = torch.rand(N, N, generator=torch.Generator().manual_seed(0)) < 0.1
    mask[5] = mask[39] = False
    p = Paged([N, N], 1, 64)
    got, _ = check_verify(p, [0, 0], [mask, torch.zeros(N, N, dtype=torch.bool)], 3, N, gate=True)
    assert (got[5] == 0).all() and (got[N:] == 0).all()
    q = torch.ones(3, 2, 64, dtype=BF16, device="cuda")
    small = Paged([2], 2, 64)
    st = i32(7)
    o = gdn.gdn_attn_prefill(small.cache(), q, i32(0, 3), small.table, i32(2), seq_status=st)  # more rows than tokens
    assert (o[0] == 0).all() and not o.isnan().any() and st.tolist() == [2]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_values_that_are_not_finite_reach_only_who_sees_them(d, bad):
    N, H, group = 45, 2, 3
    masks = [ancestors(random_tree(N, s))[1] for s in (1, 2)]
    prefix = [30, 0]
    for what in ("k", "v"):
        p = Paged([n + N for n in prefix], H, d)
        cache = p.cache()
        q = randn(generator(2), 2, N, H * group, d).to(BF16)
        bits = torch.stack([bits_of(m) for m in masks]).cuda()
        args = (bits, p.table, i32(*prefix))
        clean = gdn.gdn_attn_verify(cache, q, *args)
        node = 11
        for b in range(2):
            x = p.get(getattr(p, what), b, torch.tensor([prefix[b] + node]))
            x[:, 1, 5] = bad
            p.put(getattr(p, what), b, torch.tensor([prefix[b] + node]), x)
        got = gdn.gdn_attn_verify(cache, q, *args)
        for b in range(2):
            sees = masks[b][:, node].cuda()
            assert torch.equal(got[b][~sees], clean[b][~sees])
            assert torch.equal(got[b][:, :group], clean[b][:, :group])  # the other key head
            if what == "v":
                hit = got[b][sees][:, group:, 5].float()
                assert (hit.isnan() if bad != bad else hit == bad).all()
                hit = got[b][sees][:, group:].clone()
                hit[..., 5] = clean[b][sees][:, group:, 5]
                assert torch.equal(hit, clean[b][sees][:, group:])
    # the same in a prompt: tokens before the one with the value do not see it
    new = 100
    p = Paged([new], 1, d)
    q = randn(generator(3), new, 2, d).to(BF16)
    clean = gdn.gdn_attn_prefill(p.cache(), q, i32(0, new), p.table, i32(new))
    x = p.get(p.v, 0, torch.tensor([70]))
    x[:, 0, 3] = bad
    p.put(p.v, 0, torch.tensor([70]), x)
    got = gdn.gdn_attn_prefill(p.cache(), q, i32(0, new), p.table, i32(new))
    assert torch.equal(got[:70], clean[:70]) and not got[70:, :, 3].isfinite().any()


def test_bad_pages_are_left_out_of_tiles():
    p = Paged([300, 200], 2, 128, 16)
    p.table[0, 4], p.table[1, 12] = -1, p.k.shape[0]
    gone = [list(range(64, 80)), list(range(192, 200))]
    gen = generator(9)
    q = randn(gen, 60, 6, 128).to(BF16)
    st = i32(5, 5)
    got = gdn.gdn_attn_prefill(p.cache(), q, i32(0, 50, 60), p.table, i32(300, 200), seq_status=st)
    assert st.tolist() == [2, 2]
    for b, (a, e, n) in enumerate(((0, 50, 300), (50, 60, 200))):
        mask = causal(e - a, n)
        mask[:, gone[b]] = False
        k, v = (p.real[x][b] for x in ("k", "v"))
        ref = attend(q[a:e], k, v, mask.cuda(), 128 ** -0.5)
        close(got[a:e], ref[0], tolerance(*ref, 128, HALF))


def test_prefill_rows_of_no_sequence_are_left_alone():
    p = Paged([20, 30], 1, 64)
    q = randn(generator(1), 64, 2, 64).to(BF16)
    o = torch.full_like(q, 77.0)
    gdn.gdn_attn_prefill(p.cache(), q, i32(3, 23, 53), p.table, i32(20, 30), o=o)
    assert (o[:3] == 77).all() and (o[53:] == 77).all() and not (o[3:53] == 77).any()
    # sequences out of range are run as empty, the others are right
    want = o.clone()
    o.fill_(77.0)
    st = i32(1, 1, 1, 1)
    table, length = p.table[[0, 0, 1, 1]].contiguous(), i32(20, 20, 30, 30)
    gdn.gdn_attn_prefill(p.cache(), q, i32(3, 23, 70, 23, 53), table, length, o=o, seq_status=st)
    assert st.tolist() == [0, 2, 2, 0]
    assert torch.equal(o, want)


def test_offsets_past_32_bits():
    """pages farther apart than 2^32 bytes"""
    page, H, d, n = 16, 1, 128, 3
    far = 2 ** 31 + 64  # elements of two bytes
    big = torch.zeros(2 * far + page * d, dtype=BF16, device="cuda")
    k = big.as_strided((3, page, H, d), (far, d, d, 1))
    v = torch.randn(3, page, H, d, generator=generator(5), device="cuda").to(BF16)
    gen = generator(6)
    for i in range(n):
        k[i] = randn(gen, page, H, d).to(BF16)
    cache = gdn.GdnKvCache(k, v)
    table, length = i32(2, 0, 1).view(1, 3), i32(41)
    kk, vv = (torch.cat([x[2], x[0], x[1]])[:41].double() for x in (k, v))
    q = randn(gen, 5, 4, d).to(BF16)
    ref = attend(q[:1], kk, vv, torch.ones(1, 41, dtype=torch.bool, device="cuda"), d ** -0.5)
    close(gdn.gdn_attn_decode(cache, q[:1], table, length), ref[0], tolerance(*ref, d, TWO))
    ref = attend(q, kk, vv, causal(5, 41).cuda(), d ** -0.5)
    close(gdn.gdn_attn_prefill(cache, q, i32(0, 5), table, length), ref[0], tolerance(*ref, d, HALF))


def test_results_are_the_same_every_time_and_in_a_graph():
    lengths, N = [700, 3, 9000], 30
    p = Paged([n + N for n in lengths], 2, 128)
    cache = p.cache()
    gen = generator(1)
    q, tree_q = randn(gen, 3, 8, 128).to(BF16), randn(gen, 3, N, 8, 128).to(BF16)
    bits = torch.stack([ancestors(random_tree(N, b))[0] for b in range(3)]).cuda()
    length = i32(*lengths)
    out = [torch.empty_like(q), torch.empty_like(tree_q)]
    ws = [torch.empty(gdn.gdn_attn_workspace_bytes(kind, cache, 3, n, 8, p.table.shape[1]), dtype=torch.uint8, device="cuda")
          for kind, n in (("decode", 3), ("verify", N))]

    def run():
        gdn.gdn_attn_decode(cache, q, p.table, length, o=out[0], workspace=ws[0])
        gdn.gdn_attn_verify(cache, tree_q, bits, p.table, length, o=out[1], workspace=ws[1])

    run()
    want = [x.clone() for x in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        for x in out:
            x.zero_()
        for x in ws:
            x.fill_(255)  # nothing is kept there between calls
        if i == 2:  # lengths are read from the device: a replay follows them
            length.copy_(i32(1, 2, 3))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        run()
        assert all(torch.equal(a, b) for a, b in zip(got, out))
        if i < 2:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_on_another_stream():
    p = Paged([5000, 77], 2, 128)
    q = randn(generator(1), 2, 8, 128).to(BF16)
    length = i32(5000, 77)
    want = gdn.gdn_attn_decode(p.cache(), q, p.table, length)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        got = gdn.gdn_attn_decode(p.cache(), q, p.table, length, stream=stream)
        side.synchronize()
        assert torch.equal(got, want)


def test_empty_calls():
    p = Paged([5], 1, 64)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    assert gdn.gdn_attn_decode(p.cache(), torch.empty(0, 2, 64, dtype=BF16, device="cuda"), p.table[:0], e).shape == (0, 2, 64)
    st = i32(9)
    q = torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    assert gdn.gdn_attn_prefill(p.cache(), q, i32(0, 0), p.table, i32(5), seq_status=st).shape == (0, 2, 64)
    assert st.tolist() == [0]
    o = gdn.gdn_attn_decode(p.cache(), torch.ones(1, 2, 64, dtype=BF16, device="cuda"), p.table[:, :0], i32(0))
    assert (o == 0).all()
