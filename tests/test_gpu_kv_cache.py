"""The paged cache's writers of gdn_attn.h: append and commit, and a run of all
operators together."""
import math

import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from attn_cases import (BF16, E4M3, F32, HALF, Paged, ancestors, attend, close, generator, i32, randn,  # noqa: E402
                        random_tree, tolerance)

pytestmark = pytest.mark.gpu


def append_reference(x, weight, offset, eps, position, inv_freq, interleaved):
    x = x.double()
    if weight is not None:
        x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * (weight.double() + offset)
    if inv_freq is not None:
        angle = position.double()[:, None] * inv_freq.double()
        c, s = angle.cos()[:, None], angle.sin()[:, None]
        half = inv_freq.shape[0]
        x = x.clone()
        first, second = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
        a, b = x[..., first].clone(), x[..., second].clone()
        x[..., first], x[..., second] = a * c - b * s, b * c + a * s
    return x


def near(got, want, half):
    """Half a step of the output's type; the sums before it in fp32, and a rotation's two terms cancel: 2^-20 of the largest."""
    assert not got.double().isnan().any()
    top = want.abs().amax(-1, keepdim=True) if want.numel() else want
    err = (got.double() - want).abs() - half * want.abs() - 2.0 ** -20 * top
    assert got.numel() == 0 or err.max() <= 0, err.max()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 5, 1030])
@pytest.mark.parametrize("rot,interleaved,norm,in_dtype,dtype", [
    (0, False, False, BF16, BF16), (64, False, True, BF16, BF16), (2, True, False, F32, BF16), (32, True, True, BF16, E4M3),
    (10, False, True, F32, E4M3), (64, True, False, BF16, BF16), (34, False, False, BF16, BF16)])
def test_append(d, T, rot, interleaved, norm, in_dtype, dtype):
    H_q, H = 5, 2
    gen = generator(d + T + rot)
    p = Paged([T + 9], H, d, 16, dtype, layout=["rows", "heads", "both"][T % 3])
    before = p.k.clone().view(torch.uint8), p.v.clone().view(torch.uint8)
    rows = randn(gen, T, (2 * H_q + 2 * H) * d + 1)[:, 1:].to(in_dtype)  # query and gate of a head side by side
    q = rows[:, :2 * H_q * d].unflatten(1, (H_q, 2 * d))[..., :d]
    k, v = rows[:, 2 * H_q * d:].unflatten(1, (2 * H, d)).split([H, H], dim=1)
    w = [1 + 0.1 * randn(gen, d) for _ in range(2)] if norm else [None, None]
    position = torch.randint(0, 10 ** 6, (T,), generator=gen, device="cuda", dtype=torch.int32)
    inv = (1e4 ** (-torch.arange(0, rot, 2, device="cuda").double() / rot)).float() if rot else None
    tokens = torch.randperm(T + 9, generator=torch.Generator().manual_seed(1))[:T]
    slot = p.slots(0, tokens).to(torch.int32)
    skip = torch.arange(T, device="cuda") % 4 == 3
    slot[skip] = torch.where(slot[skip] % 2 == 0, -1, p.k.shape[0] * 16).to(torch.int32)
    got = gdn.gdn_kv_append(p.cache(), k, v, slot, position=position if rot else None, inv_freq=inv, q=q, q_weight=w[0],
                            k_weight=w[1], eps=1e-5, weight_offset=0.5 if norm else 0.0, interleaved=interleaved)
    ref = [append_reference(x, wx, 0.5, 1e-5, position, inv, interleaved) for x, wx in ((q, w[0]), (k, w[1]))]
    near(got, ref[0], HALF)
    live = (~skip).cpu()
    for pool, want, scale in ((p.k, ref[1], p.k_scale), (p.v, v.double(), p.v_scale)):
        have = p.get(pool, 0, tokens[live]).double()
        want = want[live]
        if scale is None:
            near(have, want, HALF)
        else:  # half a step of three bits; the smallest step is 2^-9
            want = (want / scale.double()[:, None]).clamp(-448, 448)
            err = (have - want).abs() - (2.0 ** -4 * want.abs()).clamp(min=2.0 ** -10) - 2.0 ** -20 * want.abs().amax(-1, keepdim=True)
            assert err.max() <= 0
    # nothing else is written
    rest = torch.ones(p.k.shape[0] * 16, dtype=torch.bool, device="cuda")
    rest[p.slots(0, tokens[live])] = False
    rest = rest.nonzero()[:, 0]
    for pool, old in ((p.k, before[0]), (p.v, before[1])):
        new = pool.view(torch.uint8)
        assert torch.equal(new[rest // 16, rest % 16], old[rest // 16, rest % 16])


def test_append_8_bit_extremes():
    """largest values are clamped, what is not finite becomes NaN, ties go to even, small values are subnormal"""
    x = torch.tensor([448.0, 464.0, 465.0, 1e30, -1e30, math.inf, -math.inf, math.nan, 0.0, 2.0 ** -9, 2.0 ** -10, 1.5 * 2.0 ** -9,
                      1.0625, 1.1875, -1.0625, 17.0], device="cuda")
    p = Paged([1], 1, 64, 16, E4M3)
    p.k_scale = p.v_scale = None
    row = x.repeat(4).view(1, 1, 64)
    gdn.gdn_kv_append(p.cache(), row, row, p.slots(0, torch.arange(1)).to(torch.int32))
    want = torch.tensor([448.0, 448.0, 448.0, 448.0, -448.0, math.nan, math.nan, math.nan, 0.0, 2.0 ** -9, 0.0, 2.0 ** -8, 1.0, 1.25,
                         -1.0, 16.0], device="cuda")
    for pool in (p.k, p.v):
        assert torch.equal(p.get(pool, 0, torch.arange(1)).float().view(4, 16).nan_to_num(-7.0), want.nan_to_num(-7.0).expand(4, 16))


def test_append_far_positions_and_in_place():
    d, T = 128, 6
    position = i32(0, 1, -5, 2 ** 31 - 1, 10 ** 6 + 1, 2 ** 30)
    inv = (5e5 ** (-torch.arange(0, d, 2, device="cuda").double() / d)).float()
    gen = generator(1)
    q, k, v = (randn(gen, T, n, d).to(BF16) for n in (3, 1, 1))
    p = Paged([T], 1, d)
    want = append_reference(q, None, 0, 0, position, inv, False)
    slot = p.slots(0, torch.arange(T)).to(torch.int32)
    assert gdn.gdn_kv_append(p.cache(), k, v, slot, position=position, inv_freq=inv, q=q, q_out=q) is q
    near(q, want, HALF)
    near(p.get(p.k, 0, torch.arange(T)), append_reference(k, None, 0, 0, position, inv, False), HALF)
    assert gdn.gdn_kv_append(p.cache(), k, v, slot, position=position, inv_freq=inv) is None  # keys and values only
    # one token, one head: strides of single tokens and heads count as dense
    one = q[:1, :1].contiguous()
    want = append_reference(one, None, 0, 0, position[1:2], inv, True)
    gdn.gdn_kv_append(p.cache(), k[:1], v[:1], slot[:1], position=position[1:2].clone(), inv_freq=inv, q=one, q_out=one, interleaved=True)
    near(one, want, HALF)
    with pytest.raises(gdn.GdnError, match="GDN_ERR_SHAPE"):
        wide = randn(gen, T, 6, d).to(BF16)[:, ::2]
        gdn._check(gdn.load_library().gdn_kv_append(
            gdn.attn.AppendDims(T, 3, 0, 0, 0, 0.0, 0.0, 0, *wide.stride()[:2], d, d, d, d), p.cache().struct, wide.data_ptr(),
            k.data_ptr(), v.data_ptr(), None, None, None, None, slot.data_ptr(), wide.data_ptr(), None))


def commit_case(lengths, N, H, d, page, dtype, layers):
    """Layers' caches on the same pages."""
    ps = [Paged([n + N for n in lengths], H, d, page, dtype, seed=i) for i in range(layers)]
    for p in ps[1:]:
        rows = [(pool, b, torch.arange(n), p.get(pool, b, torch.arange(n))) for b, n in enumerate(p.counts) for pool in (p.k, p.v)]
        p.table = ps[0].table
        for row in rows:
            p.put(*row)
    return ps


@pytest.mark.parametrize("d,H,page,dtype", [(128, 2, 16, BF16), (64, 3, 1, E4M3), (256, 2, 64, BF16), (64, 1, 8, BF16)])
@pytest.mark.parametrize("N,layers", [(1, 1), (33, 3), (256, 2), (40, 35)])
def test_commit(d, H, page, dtype, N, layers):
    lengths = [0, 1, 17, 64, 50, 200]
    B = len(lengths)
    ps = commit_case(lengths, N, H, d, page, dtype, layers)
    parents = [random_tree(N, b) for b in range(B)]
    parents[3] = list(range(-1, N - 1))  # a chain: the whole tree is one path
    accepted = [N - 1, N // 2, -1, N - 1, 0, N - 1]
    masks = [ancestors(x)[1] for x in parents]
    bits = torch.stack([ancestors(x)[0] for x in parents]).cuda()
    before = [[p.get(pool, b, torch.arange(lengths[b] + N)).clone() for pool in (p.k, p.v)] for p in ps for b in range(B)]
    st = torch.full((B,), -3, dtype=torch.int32, device="cuda")
    new = gdn.gdn_kv_commit([p.cache() for p in ps], bits, i32(*accepted), ps[0].table, i32(*lengths), seq_status=st)
    assert st.tolist() == [0] * B
    for i, p in enumerate(ps):
        for b in range(B):
            path = masks[b][accepted[b]].nonzero()[:, 0].tolist() if accepted[b] >= 0 else []
            assert new[b].item() == lengths[b] + len(path)
            for pool, old in zip((p.k, p.v), before[i * B + b]):
                want = old.clone()
                for j, node in enumerate(path):
                    want[lengths[b] + j] = old[lengths[b] + node]
                have = p.get(pool, b, torch.arange(lengths[b] + N))
                assert torch.equal(have.view(torch.uint8), want.view(torch.uint8)), (i, b)


def test_commit_reports_what_is_out_of_range():
    N, lengths = 20, [30, 30, 30, 30]
    p = Paged([n + N for n in lengths], 1, 64, 16)
    bits = torch.stack([ancestors(list(range(-1, N - 1)))[0]] * 4).cuda()
    bits[3, 5] = 0b100001  # nodes 0 and 5
    p.table[2, 2] = -1  # tokens 32 .. 47
    before = [[p.get(x, b, torch.arange(50)).clone() for x in (p.k, p.v)] for b in (0, 1, 3)]
    st, new = i32(9, 9, 9, 9), i32(0, 0, 0, 0)
    length = i32(30, 30, 30, 30)
    assert gdn.gdn_kv_commit(p.cache(), bits, i32(N, -2, 3, 5), p.table, length, new_length=new, seq_status=st) is new
    assert st.tolist() == [7, 7, 2, 0] and new.tolist() == [30, 30, 34, 32]
    for b, old in zip((0, 1, 3), before):
        for x, was in zip((p.k, p.v), old):
            want = was.clone()
            if b == 3:
                want[31] = was[35]
            assert torch.equal(p.get(x, b, torch.arange(50)), want)
    gdn.gdn_kv_commit(p.cache(), bits, i32(3, 3, 3, 3), p.table, i32(-1, 10 ** 9, 30, 30), seq_status=st)
    assert st.tolist() == [2, 2, 2, 0]
    with pytest.raises(gdn.GdnError, match="new_length"):
        gdn.gdn_kv_commit(p.cache(), bits, i32(3, 3, 3, 3), p.table, length, new_length=length)


@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_a_run_of_them_together(dtype):
    """two prompts in two steps, a tree each, its commit, and a token, against attention over the same rows in order"""
    d, H, H_q, N, page = 64, 2, 6, 24, 16
    gen = generator(3)
    p = Paged([0, 0], H, d, page, dtype, spare=24)
    p.table = torch.randperm(24, generator=torch.Generator().manual_seed(2)).to(torch.int32).view(2, 12).cuda()
    cache = p.cache()
    inv = (1e4 ** (-torch.arange(0, 32, 2, device="cuda").double() / 32)).float()
    w = [1 + 0.1 * randn(gen, d) for _ in range(2)]
    kept = [[], []]  # rows (k, v) of each sequence in order, as the cache stands for them

    def append(x, seqs, tokens, position):
        q, k, v = x.split([H_q, H, H], dim=1)
        slot = torch.cat([p.slots(b, torch.tensor([t])) for b, t in zip(seqs, tokens)]).to(torch.int32)
        q = gdn.gdn_kv_append(cache, k, v, slot, position=i32(*position), inv_freq=inv, q=q, q_weight=w[0], k_weight=w[1])
        stored = []
        for name, s in (("k", p.k_scale), ("v", p.v_scale)):
            y = torch.cat([p.get(getattr(p, name), b, torch.tensor([t])) for b, t in zip(seqs, tokens)]).double()
            stored.append(y if s is None else y * s.double()[:, None])
        return q, list(zip(*stored))

    def expect(got, q, rows, mask, weights):
        k, v = (torch.stack([r[i] for r in rows]) for i in range(2))
        ref = attend(q, k, v, mask.cuda(), d ** -0.5)
        close(got, ref[0], tolerance(*ref, d, weights))

    length = [0, 0]
    for new in ([40, 7], [21, 50]):
        seqs = [b for b in range(2) for _ in range(new[b])]
        tokens = [length[b] + i for b in range(2) for i in range(new[b])]
        q, rows = append(randn(gen, sum(new), H_q + 2 * H, d).to(BF16), seqs, tokens, tokens)
        for b, r in zip(seqs, rows):
            kept[b].append(r)
        length = [n + m for n, m in zip(length, new)]
        o = gdn.gdn_attn_prefill(cache, q, i32(0, new[0], sum(new)), p.table, i32(*length))
        at = 0
        for b in range(2):
            mask = torch.arange(length[b]) <= torch.arange(length[b] - new[b], length[b])[:, None]
            expect(o[at:at + new[b]], q[at:at + new[b]], kept[b], mask, HALF)
            at += new[b]
    parent = torch.tensor([random_tree(N, b + 5) for b in range(2)], dtype=torch.int32)
    anc, depth, _ = gdn.gdn_tree_ancestors(parent.cuda())
    seqs = [b for b in range(2) for _ in range(N)]
    tokens = [length[b] + i for b in range(2) for i in range(N)]
    position = [length[b] + depth[b, i].item() - 1 for b in range(2) for i in range(N)]
    q, rows = append(randn(gen, 2 * N, H_q + 2 * H, d).to(BF16), seqs, tokens, position)
    now = i32(*length)
    o = gdn.gdn_attn_verify(cache, q.unflatten(0, (2, N)), anc, p.table, now)
    paths = []
    for b in range(2):
        mask = ancestors(parent[b].tolist())[1]
        whole = torch.cat([torch.ones(N, length[b], dtype=torch.bool), mask], 1)
        expect(o[b], q[b * N:(b + 1) * N], kept[b] + rows[b * N:(b + 1) * N], whole, HALF)
        paths.append(mask[N - 1].nonzero()[:, 0].tolist())
        kept[b] += [rows[b * N + i] for i in paths[b]]
    now = gdn.gdn_kv_commit(cache, anc, i32(N - 1, N - 1), p.table, now)
    length = [n + len(x) for n, x in zip(length, paths)]
    assert now.tolist() == length
    q, rows = append(randn(gen, 2, H_q + 2 * H, d).to(BF16), [0, 1], length, length)
    o = gdn.gdn_attn_decode(cache, q, p.table, now + 1)
    for b in range(2):
        kept[b].append(rows[b])
        expect(o[b:b + 1], q[b:b + 1], kept[b], torch.ones(1, len(kept[b]), dtype=torch.bool), HALF * HALF)
