"""More of the operators around the tree verify on the GPU: norms over rows
that are aligned to their elements only, and the walk and the chunks of
gdn_prefill on either side of the sizes that choose between them.

Tolerances as for the other tests of these operators (a row's arithmetic does
not depend on its alignment).
"""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from test_gpu_layer import BF16, CHUNK_TOL, F32, FP32_TOL, LINEAR_TOL, check, gpu, make, rel, rms, run_prefill, say  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def at_offset(x, off):
    """A copy of x [T][n] as a slice that starts `off` elements into wider rows of odd length."""
    wide = torch.full((x.shape[0], (x.shape[1] + off) | 1), 7.0, dtype=x.dtype, device=x.device)
    view = wide[:, off:off + x.shape[1]]
    view.copy_(x)
    return view, wide


@pytest.mark.parametrize("D", [1, 5, 8, 64, 101, 1001, 4096, 4097, 5119, 8199, 16383])
@pytest.mark.parametrize("off", [1, 3, 4, 7])
def test_add_norm_of_unaligned_rows(D, off):
    gen = torch.Generator().manual_seed(D + off)
    randn = lambda *n: torch.randn(*n, generator=gen).cuda()  # noqa: E731
    w, p, c = randn(D), randn(D), randn(D)
    for x_dt, r_dt, y_dt, post, chan in ((BF16, F32, BF16, p, c), (BF16, BF16, F32, None, None), (F32, BF16, BF16, p, None)):
        x, _ = at_offset(randn(5, D).to(x_dt), off)
        r, _ = at_offset((3 * randn(5, D)).to(r_dt), off)
        h, h_wide = at_offset(torch.zeros(5, D, dtype=r_dt, device="cuda"), off)
        y, y_wide = at_offset(torch.zeros(5, D, dtype=y_dt, device="cuda"), off)
        X, R, W, P, C = (a.cpu().double() for a in (x, r, w, p, c))
        gdn.gdn_add_norm(x, r, w, scale=0.7, chan_scale=chan, post_weight=post, h=h, y=y)
        z = rms(X) * P if post is not None else X
        want = R + 0.7 * (z * C if chan is not None else z)
        check(h, want, FP32_TOL, f"h, D {D} at {off}")
        check(y, rms(want) * W, FP32_TOL, "y")
        for wide in (h_wide, y_wide):  # nothing beside the rows is written
            assert (wide[:, :off] == 7.0).all() and (wide[:, off + D:] == 7.0).all()
        gdn.gdn_add_norm(x, r, w, scale=0.7, chan_scale=chan, post_weight=post, h=r, y=y)
        assert torch.equal(r, h)  # in place of the residual


@pytest.mark.parametrize("d", [1, 5, 8, 33, 64, 80, 127, 128, 200, 511, 513])
@pytest.mark.parametrize("off", [1, 3, 7])
@pytest.mark.parametrize("H", [1, 7])
def test_gated_norm_of_unaligned_rows(H, d, off):
    gen = torch.Generator().manual_seed(H + d + off)
    randn = lambda *n: torch.randn(*n, generator=gen).cuda()  # noqa: E731
    w = randn(d)
    for o_dt, z_dt, y_dt in ((F32, BF16, BF16), (BF16, BF16, F32), (BF16, F32, BF16)):
        o, _ = at_offset(randn(9, H * d).to(o_dt), off)
        z, _ = at_offset(randn(9, H * d).to(z_dt), off)
        y, wide = at_offset(torch.zeros(9, H * d, dtype=y_dt, device="cuda"), off)
        gdn.gdn_gated_norm(*(x.unflatten(1, (H, d)) for x in (o, z)), w, y=y.unflatten(1, (H, d)))
        O, Z = (x.cpu().double().unflatten(1, (H, d)) for x in (o, z))
        check(y, (rms(O) * w.cpu().double() * torch.nn.functional.silu(Z)).flatten(1), FP32_TOL, f"H {H} d {d} at {off}")
        assert (wide[:, :off] == 7.0).all() and (wide[:, off + H * d:] == 7.0).all()


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128)])
def test_walk_and_chunks_agree(dk, dv):
    """8 tokens per sequence on average are walked, one token more makes chunks of them."""
    lengths = [1, 0, 29, 2, 8, 8]
    extra = lengths + [1]
    n = sum(lengths)
    assert n == 8 * len(lengths) and n + 17 > 8 * len(extra)
    d = make(n + 17, 2, 4, dk, dv, slots=7, seed=3)
    o1, S1 = run_prefill({a: x if a == "S" else x[:n].contiguous() for a, x in d.items()}, lengths)
    o2, S2 = run_prefill(d, lengths + [17])
    assert rel(o1, o2[:n]) <= CHUNK_TOL and rel(S1[:6], S2[:6]) <= CHUNK_TOL


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B", [1, 2, 8, 9])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_walk_of_few_and_many_rows(B, dk, dv, dtype):
    """Both splits of a state row over lanes, sequences around the four tokens that are loaded ahead."""
    lengths = [[3, 4, 5, 0, 8, 7, 1, 2, 9][b] for b in range(B)]
    d = make(sum(lengths), 8, 32, dk, dv, dtype=dtype, slots=B, seed=B)
    run_prefill(d, lengths, has=[b % 2 for b in range(B)], qk_l2norm=True, q_scale=0.125, o_dtype=F32)


def test_chunks_of_short_sequences():
    """Sequences of a few tokens beside one long enough for all of them to be cut into chunks."""
    lengths = [1, 2, 3, 16, 17, 63, 0, 64, 65, 200]
    say(f"[prefill] {lengths}")
    d = make(sum(lengths), slots=10, seed=1)
    run_prefill(d, lengths, has=[1, 0] * 5, o_dtype=F32)


def test_a_decode_step_in_a_graph():
    """norm, projection, decode, gated norm and projection captured once and replayed: every replay equals the eager step
    bit for bit, from the same state, with eager work of other sizes between the replays."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    randn = lambda *n: torch.randn(*n, generator=gen, device="cuda")  # noqa: E731
    B, D, Hk, Hv, dh = 9, 200, 2, 4, 64
    x, h = randn(B, D).to(BF16), randn(B, D)
    w, wo, norm, head = randn((2 * Hk + 2 * Hv) * dh, D).to(BF16), randn(D, Hv * dh).to(BF16), randn(D), randn(dh)
    g, beta, S = -torch.rand(B, Hv, device="cuda"), torch.rand(B, Hv, device="cuda"), randn(B, Hv, dh, dh)
    S0 = S.clone()

    def step():
        y, r = gdn.gdn_add_norm(x, h, norm)
        q, k, v, z = gdn.gdn_linear(y, w).unflatten(1, (-1, dh)).split([Hk, Hk, Hv, Hv], dim=1)
        o = gdn.gdn_decode(q, k, v, g, beta, S, qk_l2norm=True, o_dtype=F32)
        return gdn.gdn_linear(gdn.gdn_gated_norm(o, z, head).flatten(1), wo, residual=r, y_dtype=F32)

    want = step().clone()
    want_S = S.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        S.copy_(S0)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(S, want_S), i
        gdn.gdn_linear(randn(300 + i, D).to(BF16), w)
        torch.cuda.synchronize()


# one for each tile and for 256 x 256 tiles with the last ones in quarters
@pytest.mark.parametrize("M,N", [(40, 300), (300, 900), (130, 5000), (777, 4096), (1100, 4100), (4300, 4096)])
@pytest.mark.parametrize("K", [8, 56, 64, 72, 200, 264, 440])
def test_linear_ends_of_k(M, N, K):
    """K in whole pieces of 8 but not in whole steps of 64, the rows slices of wider ones that hold NaN beside them."""
    if M > 4000 and K not in (72, 200):
        pytest.skip("two of the largest are enough")
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    wide = [torch.full((n, K + 16), float("nan"), dtype=BF16, device="cuda") for n in (M, N)]
    x, w = (t[:, 8:8 + K] for t in wide)
    x.copy_(torch.randn(M, K, generator=gen, device="cuda"))
    w.copy_(torch.randn(N, K, generator=gen, device="cuda") * K ** -0.5)
    y = gdn.gdn_linear(x, w, y_dtype=F32)
    want = x.double().contiguous() @ w.double().t().contiguous()
    check(y, want, LINEAR_TOL, f"{M} x {N} x {K}")
    x[3, K - 1] = float("inf")  # the last element: its row alone, no NaN from what was cleared
    y2 = gdn.gdn_linear(x, w, y_dtype=F32)
    assert torch.isinf(y2[3]).all()
    assert torch.equal(y2[:3], y[:3]) and torch.equal(y2[4:], y[4:])


def test_more_workgroups_than_one_grid_dimension_holds():
    """More than 2^20 rows, and more than 2^20 workgroups of the chunked delta rule: sequences of no tokens beside a few."""
    T, D = (1 << 20) + 3, 8
    x = torch.randn(T, D, device="cuda")
    y, _ = gdn.gdn_add_norm(x, None, torch.ones(D, device="cuda"), y_dtype=F32)
    check(y[-5:], rms(x[-5:].cpu().double()), FP32_TOL, "the last rows")
    check(y[(1 << 20) - 2:(1 << 20) + 2], rms(x[(1 << 20) - 2:(1 << 20) + 2].cpu().double()), FP32_TOL, "around 2^20")

    B, H = 20000, 16
    n = 8 * B + 64
    d = make(200, 1, H, 64, 64, slots=2, seed=2)
    far = [B - 3, B - 1]
    q, k, v, g, beta = (torch.zeros(n, *d[a].shape[1:], dtype=d[a].dtype, device="cuda") for a in ("q", "k", "v", "g", "beta"))
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[far[0] + 1:] += 120
    cu[far[1] + 1:] += 80
    for t, a in ((q, "q"), (k, "k"), (v, "v"), (g, "g"), (beta, "beta")):
        t[:200] = d[a]
    slot = torch.full((B,), -1, dtype=torch.int32)
    slot[far] = torch.tensor([0, 1], dtype=torch.int32)
    S = d["S"].clone()
    o = gdn.gdn_prefill(q, k, v, g, beta, cu.cuda(), S, slot=slot.cuda(), o_dtype=F32)
    want, S2 = run_prefill(d, [120, 80])
    assert torch.equal(o[:200], want) and torch.equal(S, S2)
