"""The operators around the tree verify (gdn_layer.h) on the GPU, against
plain 64-bit implementations of their definitions.

Tolerances, in rel-L2 = |x - y| / |y| over a whole output:
 - a bf16 output: each element is rounded once to 8 significant bits, off by
   at most 2^-8 of itself, so 2^-8 = 3.9e-3, plus the fp32 bound below;
 - an fp32 output or state: the operands of the chunked path are split into
   two bf16 parts or more, off by at most 2^-16 of an element: 2^-16 = 1.5e-5
   (their errors are independent, so sums of them stay below).  The token by
   token path and the norms work in plain fp32: 2e-6, some 30 roundings of
   2^-24; matrix products add K terms in fp32, at most sqrt(K) 2^-24 at random
   signs, 4e-6 at K = 4096, and the gate functions a few more: 1e-5.
"""
import sys

import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
CHUNK_TOL, FP32_TOL, LINEAR_TOL = 2.0 ** -16, 2e-6, 1e-5


def say(msg):
    print(msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.fail("no GPU visible: GPU tests need an MI355X")
    gdn.load_library()


def rel(x, y):
    x, y = x.detach().cpu().double(), y.detach().cpu().double()
    assert torch.isfinite(x).all()
    n = y.norm()
    return float((x - y).norm() / n) if n > 0 else float((x - y).norm())


def check(x, y, tol, what):
    assert x.shape == y.shape, what
    if x.dtype == BF16:
        tol = tol + 2.0 ** -8
    r = rel(x, y)
    say(f"  {what}: rel-L2 {r:.2e} (tolerance {tol:.2e})")
    assert r <= tol, what


# ----------------------------------------------------------------------------
# the delta rule
# ----------------------------------------------------------------------------

def recurrence(q, k, v, g, beta, S, q_scale=1.0, l2norm=False, eps=1e-6):
    """o [n][Hv][dv] and the final state of one sequence, token by token in 64
    bits on the CPU; S [Hv][dv][dk]."""
    q, k, v, g, beta, S = (x.detach().cpu().double() for x in (q, k, v, g, beta, S))
    if l2norm:
        q = q / (q.square().sum(-1, keepdim=True) + eps).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + eps).sqrt()
    r = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(r, 1) * q_scale, k.repeat_interleave(r, 1)
    o = torch.zeros(v.shape, dtype=torch.double)
    for t in range(v.shape[0]):
        S = torch.exp(g[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - (S * k[t][:, None, :]).sum(-1))
        S = S + u[..., None] * k[t][:, None, :]
        o[t] = (S * q[t][:, None, :]).sum(-1)
    return o, S


def make(T, Hk=2, Hv=4, dk=128, dv=128, dtype=BF16, seed=0, unit=True, slots=1, rate=0.7):
    gen = torch.Generator().manual_seed(seed)
    randn = lambda *n: torch.randn(*n, generator=gen)  # noqa: E731
    q, k = randn(T, Hk, dk), randn(T, Hk, dk)
    if unit:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    d = dict(q=q.to(dtype), k=k.to(dtype), v=randn(T, Hv, dv).to(dtype),
             g=-rate * torch.rand(T, Hv, generator=gen) * torch.linspace(0.02, 2, Hv),
             beta=torch.sigmoid(randn(T, Hv)), S=0.5 * randn(slots, Hv, dv, dk))
    return {n: x.cuda() for n, x in d.items()}


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run_prefill(d, lengths, slot=None, has=None, start=0, o_dtype=F32, **kw):
    """Runs and checks one packed batch; returns (o, S)."""
    cu = [start]
    for n in lengths:
        cu.append(cu[-1] + n)
    S0, S = d["S"].clone(), d["S"].clone()
    status = torch.full((len(lengths),), 77, dtype=torch.int32, device="cuda")
    o = torch.full(d["v"].shape, 7.0, dtype=o_dtype, device="cuda")
    gdn.gdn_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], i32(*cu), S,
                    slot=None if slot is None else i32(*slot), has_state=None if has is None else i32(*has),
                    o=o, seq_status=status, **kw)
    torch.cuda.synchronize()
    assert status.tolist() == [0] * len(lengths)
    want_o, want_S = torch.full(d["v"].shape, 7.0, dtype=torch.double), S0.cpu().double()
    kw = {"l2norm" if a == "qk_l2norm" else a: x for a, x in kw.items() if a in ("q_scale", "qk_l2norm")}
    for b, n in enumerate(lengths):
        at = b if slot is None else slot[b]
        kept = 0 <= at < S0.shape[0]
        init = S0[at] if kept and (has is None or has[b]) else torch.zeros_like(S0[0])
        x = slice(cu[b], cu[b + 1])
        want_o[x], end = recurrence(*(d[a][x] for a in ("q", "k", "v", "g", "beta")), init, **kw)
        if kept:
            want_S[at] = end
    check(o, want_o, CHUNK_TOL, f"o, lengths {lengths}")
    check(S, want_S, CHUNK_TOL, "S")
    # per sequence too, so that a short one cannot hide behind a long one
    for b, n in enumerate(lengths):
        if n:
            check(o[cu[b]:cu[b + 1]], want_o[cu[b]:cu[b + 1]], 2 * CHUNK_TOL, f"o of sequence {b} ({n} tokens)")
    for x in (slice(0, start), slice(cu[-1], None)):  # tokens of no sequence
        assert (o[x] == 7.0).all()
    return o, S


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 449])
def test_prefill_lengths(n, dtype):
    say(f"[prefill] one sequence of {n} tokens, {dtype}")
    run_prefill(make(n, dtype=dtype, seed=n), [n])


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (3, 3), (2, 6), (1, 4), (2, 10)])
def test_prefill_heads(Hk, Hv, dk, dv):
    say(f"[prefill] {Hk} key and {Hv} value heads, d {dk} {dv}")
    run_prefill(make(150, Hk, Hv, dk, dv, seed=Hk + Hv, slots=2), [70, 80], o_dtype=BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_packed(dtype):
    say(f"[prefill] ragged batch with empty sequences, slots and fresh states, {dtype}")
    lengths = [5, 0, 64, 1, 130, 0, 63, 257, 2, 0]
    d = make(sum(lengths) + 9, dtype=dtype, seed=3, slots=12, unit=False)
    run_prefill(d, lengths, slot=[11, 3, -1, 5, 7, 0, 2, 9, 12, 4], has=[1, 0, 1, 0, 1, 1, 0, 1, 1, 0], start=4,
                q_scale=0.25, qk_l2norm=True)


def test_prefill_many_sequences():
    say("[prefill] 300 sequences of 0 to 4 tokens")
    gen = torch.Generator().manual_seed(0)
    lengths = torch.randint(0, 5, (300,), generator=gen).tolist()
    run_prefill(make(sum(lengths), 1, 2, 64, 64, seed=4, slots=300), lengths)


def test_prefill_without_a_pool():
    d = make(100, seed=5)
    d["S"] = d["S"][:0]
    o = gdn.gdn_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], i32(0, 100), d["S"], slot=i32(-1), o_dtype=F32)
    want, _ = recurrence(*(d[a] for a in ("q", "k", "v", "g", "beta")), torch.zeros(4, 128, 128))
    check(o, want, CHUNK_TOL, "o from zero, state dropped")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_slices_of_one_projection(dtype):
    """q, k and v as slices of wider rows, the value rows broadcast over tokens"""
    d = make(100, seed=6, dtype=dtype)
    rows = torch.randn(100, 2 * 2 * 128 + 4 * 128 + 64, device="cuda").to(dtype)
    wide = dict(d, q=rows[:, :256].unflatten(1, (2, 128)), k=rows[:, 256:512].unflatten(1, (2, 128)),
                v=rows[:, 512:1024].unflatten(1, (4, 128)))
    run_prefill(wide, [40, 60], slot=[-1, 0], qk_l2norm=True)
    run_prefill(dict(d, v=d["v"][:1].expand(100, 4, 128)), [100])


def test_prefill_in_two_parts_equals_one():
    d = make(300, seed=7)
    S1 = d["S"].clone()
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    o1 = gdn.gdn_prefill(*args, i32(0, 300), S1, o_dtype=F32)
    S2 = d["S"].clone()
    a = gdn.gdn_prefill(*(x[:77] for x in args), i32(0, 77), S2, o_dtype=F32)
    b = gdn.gdn_prefill(*(x[77:] for x in args), i32(0, 223), S2, o_dtype=F32)
    check(torch.cat([a, b]), o1, 2 * CHUNK_TOL, "o in two parts")
    check(S2, S1, 2 * CHUNK_TOL, "S in two parts")


@pytest.mark.parametrize("what", ["no decay", "hard decay", "resets", "beta one, one key", "beta zero", "growth"])
def test_prefill_extreme_gates(what):
    d = make(200, seed=8)
    if what == "no decay":
        d["g"].zero_()
    elif what == "hard decay":  # decays far below the smallest fp32 inside a chunk
        d["g"].mul_(200.0)
    elif what == "resets":  # alpha = 0 now and then, gentle decay otherwise
        d["g"][::7] = -float("inf")
    elif what == "beta one, one key":
        d["beta"].fill_(1.0)
        d["k"].copy_(d["k"][:1].expand_as(d["k"]).clone())
    elif what == "beta zero":
        d["beta"].zero_()
    else:
        d["g"].fill_(0.05)
    say(f"[prefill] {what}")
    run_prefill(d, [200])


@pytest.mark.parametrize("name", ["v", "k", "g", "beta", "q"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("at", [0, 20, 63, 64, 100])
def test_prefill_non_finite_stays_behind(name, bad, at):
    """a value that is not finite reaches neither earlier tokens nor other
    sequences, and reaches what depends on it"""
    d = make(260, seed=9, slots=2)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    cu = i32(0, 130, 260)
    S1 = d["S"].clone()
    o1 = gdn.gdn_prefill(*args, cu, S1, o_dtype=F32)
    x = d[name].clone()
    if x.dim() == 3:
        x[at, 1, 3] = bad
    else:
        x[at, 2] = bad
    S2 = d["S"].clone()
    o2 = gdn.gdn_prefill(*[x if a == name else y for a, y in zip(("q", "k", "v", "g", "beta"), args)], cu, S2,
                         o_dtype=F32)
    assert torch.isfinite(o2[:at]).all() and rel(o2[:at], o1[:at]) <= CHUNK_TOL
    assert torch.equal(o2[130:], o1[130:]) and torch.equal(S2[1], S1[1])
    if name == "v":  # value head 1, element 3 only
        assert not torch.isfinite(o2[at, 1, 3])
        rest = torch.ones_like(o2, dtype=torch.bool)
        rest[:, 1, 3] = False
        assert rel(o2[rest], o1[rest]) <= CHUNK_TOL
        assert not torch.isfinite(S2[0, 1, 3]).any() and torch.isfinite(S2[0, 1, 4]).all()
    elif name == "q":  # one token of the value heads of key head 1
        assert not torch.isfinite(o2[at, 2:]).any()
        o2[at, 2:] = o1[at, 2:]
        assert rel(o2, o1) <= CHUNK_TOL and rel(S2, S1) <= CHUNK_TOL
    else:
        assert not torch.isfinite(o2[at:130, 2]).any() or bad == float("inf") and name == "g"
        assert not torch.isfinite(S2[0, 2]).all()
        assert torch.isfinite(o2[:, :2]).all() if name == "k" else torch.isfinite(o2[:, [0, 1, 3]]).all()


def test_prefill_bad_offsets_are_reported():
    """sequences whose offsets are not 0 <= start <= end <= T run as empty; the others are right"""
    for dtype in (BF16, F32):
        d = make(200, seed=10, dtype=dtype, slots=4)
        S = d["S"].clone()
        status = i32(9, 9, 9, 9)
        args = [d[a] for a in ("q", "k", "v", "g", "beta")]
        o = gdn.gdn_prefill(*args, i32(0, 90, 60, 150, 201), S, o_dtype=F32, seq_status=status)
        torch.cuda.synchronize()
        assert status.tolist() == [0, 2, 0, 2]
        want, end = recurrence(*(x[:90] for x in args), d["S"][0])
        check(o[:60], want[:60], CHUNK_TOL, "o of the first sequence, where no other overlaps it")
        check(S[0], end, CHUNK_TOL, "S of the first sequence")
        assert torch.equal(S[1], d["S"][1]) and torch.equal(S[3], d["S"][3])
        status = i32(9)
        gdn.gdn_prefill(*args, i32(-5, 100), S[:1], seq_status=status)
        assert status.tolist() == [2]


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prefill_is_deterministic_and_ignores_its_workspace(dtype):
    d = make(700, 4, 8, seed=11, dtype=dtype, slots=3)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    cu = i32(0, 300, 301, 700)
    need = gdn.gdn_prefill_workspace_bytes(d["q"], d["v"], cu)
    runs = []
    for fill in (0, 255, 127):
        ws = torch.full((max(need, 1),), fill, dtype=torch.uint8, device="cuda")
        S = d["S"].clone()
        runs.append((gdn.gdn_prefill(*args, cu, S, o_dtype=F32, workspace=ws), S))
    for o, S in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(S, runs[0][1])


def test_prefill_on_another_stream():
    d = make(500, seed=12)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    S1, S2 = d["S"].clone(), d["S"].clone()
    o1 = gdn.gdn_prefill(*args, i32(0, 500), S1)
    cu = i32(0, 500)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o2 = gdn.gdn_prefill(*args, cu, S2, stream=side)
    junk = [torch.full((1 << 22,), 3.0, device="cuda") for _ in range(8)]  # would reuse memory freed too early
    side.synchronize()
    assert torch.equal(o1, o2) and torch.equal(S1, S2) and len(junk) == 8


def test_prefill_in_a_graph():
    """captured and replayed several times with eager work between the replays"""
    d = make(300, seed=13)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    cu = i32(0, 100, 300)
    d["S"] = d["S"].repeat(2, 1, 1, 1).contiguous()
    S = d["S"].clone()
    o = torch.empty(300, 4, 128, device="cuda")
    ws = torch.empty(gdn.gdn_prefill_workspace_bytes(d["q"], d["v"], cu), dtype=torch.uint8, device="cuda")
    gdn.gdn_prefill(*args, cu, S, o=o, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.gdn_prefill(*args, cu, S, o=o, workspace=ws)
    for i in range(4):
        d["v"].mul_(0.9)
        S.copy_(d["S"])
        graph.replay()
        torch.cuda.synchronize()
        S1 = d["S"].clone()
        o1 = gdn.gdn_prefill(*args, cu, S1, o_dtype=F32)
        assert torch.equal(o, o1) and torch.equal(S, S1)


def test_prefill_state_feeds_the_tree_verify():
    """the state of a prompt is the S0 of gdn_tree_verify: verifying a chain
    equals running its tokens through the prefill"""
    d = make(100 + 32, seed=14)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    S = d["S"].clone()
    gdn.gdn_prefill(*(x[:100] for x in args), i32(0, 100), S)
    parent = torch.arange(-1, 31, dtype=torch.int32, device="cuda")[None]
    o, ctx = gdn.verify(*(x[None, 100:].contiguous() for x in args), parent, S)
    committed = gdn.gdn_commit_path(ctx, i32(31))
    o2 = gdn.gdn_prefill(*(x[100:] for x in args), i32(0, 32), S, o_dtype=F32)
    assert rel(o[0], o2) <= 1e-3 and rel(committed, S) <= 1e-3


# ----------------------------------------------------------------------------
# single tokens
# ----------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("B,Hk,Hv", [(1, 1, 1), (5, 2, 6), (130, 2, 4)])
def test_decode(B, Hk, Hv, dk, dv, dtype):
    say(f"[decode] B {B} heads {Hk} {Hv} d {dk} {dv} {dtype}")
    d = make(B, Hk, Hv, dk, dv, dtype, seed=B, unit=False, slots=B + 3)
    gen = torch.Generator().manual_seed(B)
    slot = torch.randperm(B + 3, generator=gen)[:B].tolist()
    slot[B // 2] = [-1, B + 3, 0][B % 3] if B > 1 else slot[0]
    if B > 1 and slot.count(0) > 1:
        slot[slot.index(0)] = -1
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    S = d["S"].clone()
    o = gdn.gdn_decode(*args, S, slot=i32(*slot), q_scale=0.3, qk_l2norm=True, o_dtype=F32)
    want_o, want_S = torch.zeros(B, Hv, dv, dtype=torch.double), d["S"].cpu().double()
    for b, at in enumerate(slot):
        if 0 <= at < B + 3:
            want_o[b:b + 1], want_S[at] = recurrence(*(x[b:b + 1] for x in args), d["S"][at], 0.3, True)
    check(o, want_o, FP32_TOL, "o")
    check(S, want_S, FP32_TOL, "S")
    idle = [b for b, at in enumerate(slot) if not 0 <= at < B + 3]
    assert (o[idle] == 0).all()
    S = d["S"].clone()
    check(gdn.gdn_decode(*args, S, slot=i32(*slot), q_scale=0.3, qk_l2norm=True, o_dtype=BF16), want_o, FP32_TOL, "o bf16")


def test_decode_follows_prefill():
    """tokens one by one equal the same tokens as a prompt"""
    d = make(80, seed=20)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    S1, S2 = d["S"].clone(), d["S"].clone()
    o1 = gdn.gdn_prefill(*args, i32(0, 80), S1, o_dtype=F32)
    o2 = torch.cat([gdn.gdn_decode(*(x[t:t + 1] for x in args), S2, o_dtype=F32) for t in range(80)])
    check(o2, o1, CHUNK_TOL, "o")
    check(S2, S1, CHUNK_TOL, "S")


def test_decode_past_32_bit_offsets():
    """a pool of more than 2^31 elements"""
    slots = (1 << 31) // (4 * 128 * 128) + 3
    d = make(2, seed=21)
    S = torch.empty(slots, 4, 128, 128, device="cuda")
    at = [slots - 1, slots - 2]
    S[at] = torch.randn(2, 4, 128, 128, device="cuda")
    first = S[at].clone()
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    o = gdn.gdn_decode(*args, S, slot=i32(*at), o_dtype=F32)
    for b in range(2):
        want, end = recurrence(*(x[b:b + 1] for x in args), first[b])
        check(o[b:b + 1], want, FP32_TOL, "o")
        check(S[at[b]], end, FP32_TOL, "S")


# ----------------------------------------------------------------------------
# norms
# ----------------------------------------------------------------------------

def rms(x, eps=1e-6):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


@pytest.mark.parametrize("D", [1, 7, 8, 64, 65, 128, 520, 1000, 2048, 4096, 5120, 8192, 12345, 16384])
@pytest.mark.parametrize("T", [1, 3, 70])
@pytest.mark.parametrize("x_dtype,r_dtype,y_dtype", [(BF16, BF16, BF16), (F32, F32, F32), (BF16, F32, BF16)])
def test_add_norm(T, D, x_dtype, r_dtype, y_dtype):
    gen = torch.Generator().manual_seed(T + D)
    randn = lambda *n: torch.randn(*n, generator=gen).cuda()  # noqa: E731
    x, r, w, p, c = randn(T, D).to(x_dtype), (3 * randn(T, D)).to(r_dtype), randn(D), randn(D), randn(D)
    X, R, W, P, C = (a.cpu().double() for a in (x, r, w, p, c))
    for post, chan, res, off in ((None, None, True, 0.0), (p, c, True, 1.0), (p, None, False, 0.0)):
        y, h = gdn.gdn_add_norm(x, r if res else None, w, scale=0.7, chan_scale=chan, post_weight=post,
                                weight_offset=off, y_dtype=y_dtype)
        z = rms(X) * (P + off) if post is not None else X
        want_h = (R if res else 0) + 0.7 * (z * C if chan is not None else z)
        check(h, want_h, FP32_TOL, f"h T {T} D {D}")
        check(y, rms(want_h) * (W + off), FP32_TOL, "y")


def test_add_norm_in_place_and_strided():
    x, r, w = torch.randn(9, 600, device="cuda"), torch.randn(9, 600, device="cuda"), torch.ones(256, device="cuda")
    for lo in (0, 44):  # 16-byte pieces, and rows of no alignment (an odd stride)
        for width in (600, 599):
            base = torch.randn(9, width, device="cuda")
            res = base[:, lo:lo + 256]
            want = res.cpu().double() + x[:, 8:264].cpu().double()
            out = torch.zeros(9, 300, device="cuda")
            y, h = gdn.gdn_add_norm(x[:, 8:264], res, w, h=res, y=out[:, :256], y_dtype=F32)
            assert h.data_ptr() == res.data_ptr()
            check(res, want, FP32_TOL, "h in place")
            check(out[:, :256], rms(want), FP32_TOL, "y in wider rows")
            assert (out[:, 256:] == 0).all()


def test_norm_of_zero_rows_and_non_finite_rows():
    x = torch.randn(4, 256, device="cuda")
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    y, h = gdn.gdn_add_norm(x, None, torch.ones(256, device="cuda"), y_dtype=F32)
    assert torch.isfinite(y[:2]).all() and (y[1] == 0).all()
    assert not torch.isfinite(y[2]).all() and torch.isnan(y[3]).all()


@pytest.mark.parametrize("d", [1, 5, 8, 33, 64, 72, 80, 128, 256, 512, 520, 1000])
@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (65, 32)])
@pytest.mark.parametrize("gate", ["silu", "sigmoid"])
def test_gated_norm(T, H, d, gate):
    gen = torch.Generator().manual_seed(T + H + d)
    o = torch.randn(T, H, d, generator=gen).cuda()
    wide = torch.randn(T, 2 * H * d + 8, generator=gen).cuda()
    w = torch.randn(d, generator=gen).cuda()
    lo = (H * d + 7) // 8 * 8  # a slice of a projection, 16-byte aligned
    for o_dt, z_dt, y_dt in ((F32, BF16, BF16), (BF16, BF16, F32), (F32, F32, F32)):
        z = wide.to(z_dt)[:, lo:lo + H * d].unflatten(1, (H, d))
        y = gdn.gdn_gated_norm(o.to(o_dt), z, w, gate=gate, y_dtype=y_dt)
        Z = z.cpu().double()
        want = rms(o.to(o_dt).cpu().double()) * w.cpu().double() * torch.sigmoid(Z) * (Z if gate == "silu" else 1)
        check(y, want, FP32_TOL, f"T {T} H {H} d {d} {gate}")


def test_gated_norm_in_place_and_large_gates():
    o = torch.randn(10, 4, 128, device="cuda")
    z = torch.randn(10, 4, 128, device="cuda") * 60  # far tails of the gate
    w = torch.ones(128, device="cuda")
    want = rms(o.cpu().double()) * torch.nn.functional.silu(z.cpu().double())
    y = gdn.gdn_gated_norm(o, z, w, y=o, y_dtype=F32)
    assert y.data_ptr() == o.data_ptr()
    check(o, want, FP32_TOL, "y in place of o")


# ----------------------------------------------------------------------------
# projections
# ----------------------------------------------------------------------------

def linear_case(M, N, K, act="none", bias=True, res=None, y_dtype=F32, scale=0.5, seed=0):
    gen = torch.Generator().manual_seed(seed + M + N + K)
    x = torch.randn(M, K, generator=gen).to(BF16).cuda()
    w = (torch.randn(N, K, generator=gen) * K ** -0.5).to(BF16).cuda()
    b = torch.randn(N, generator=gen).cuda() if bias else None
    r = torch.randn(M, N, generator=gen).to(res).cuda() if res is not None else None
    y = gdn.gdn_linear(x, w, bias=b, act=act, residual=r, scale=scale, y_dtype=y_dtype)
    z = x.cpu().double() @ w.cpu().double().t().contiguous()
    if bias:
        z = z + b.cpu().double()
    z = {"none": lambda a: a, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "sigmoid": torch.sigmoid}[act](z) * scale
    if r is not None:
        z = z + r.cpu().double()
    check(y, z, LINEAR_TOL, f"M {M} N {N} K {K} {act}")


@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 33, 64, 65, 100, 129, 257, 300])
@pytest.mark.parametrize("N,K", [(16, 64), (1, 1), (130, 100), (513, 512), (257, 129), (1000, 4096), (72, 8)])
def test_linear_shapes(M, N, K):
    linear_case(M, N, K)


@pytest.mark.parametrize("M,N,K", [(1024, 1536, 512), (515, 769, 264), (2048, 256, 1024)])
def test_linear_large(M, N, K):
    linear_case(M, N, K, act="silu", res=BF16, y_dtype=BF16)


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("res", [None, BF16, F32])
@pytest.mark.parametrize("M", [3, 150])
def test_linear_epilogue(M, act, bias, res):
    linear_case(M, 200, 96, act=act, bias=bias, res=res, y_dtype=BF16)
    linear_case(M, 200, 96, act=act, bias=bias, res=res, scale=1.0)


def test_linear_without_inputs():
    """K = 0 leaves bias, activation and residual; M = 0 and N = 0 nothing"""
    b, r = torch.randn(5, device="cuda"), torch.randn(3, 5, device="cuda")
    y = gdn.gdn_linear(torch.empty(3, 0, dtype=BF16, device="cuda"), torch.empty(5, 0, dtype=BF16, device="cuda"),
                       bias=b, residual=r, y_dtype=F32)
    assert torch.equal(y, r + b)
    assert gdn.gdn_linear(torch.empty(0, 8, dtype=BF16, device="cuda"), torch.empty(5, 8, dtype=BF16, device="cuda")).shape == (0, 5)
    assert gdn.gdn_linear(torch.empty(2, 8, dtype=BF16, device="cuda"), torch.empty(0, 8, dtype=BF16, device="cuda")).shape == (2, 0)


@pytest.mark.parametrize("M", [1, 5, 200])
def test_linear_strides_and_in_place(M):
    gen = torch.Generator().manual_seed(M)
    xw = torch.randn(M, 700, generator=gen).to(BF16).cuda()
    ww = torch.randn(90, 777, generator=gen).to(BF16).cuda()
    x, w = xw[:, 8:264], ww[:, :256]  # aligned and unaligned rows
    yw = torch.randn(M, 131, generator=gen).cuda()
    y = yw[:, :90]
    want = y.cpu().double() + x.cpu().double() @ w.cpu().double().t().contiguous()
    rest = yw[:, 90:].clone()
    gdn.gdn_linear(x, w, residual=y, y=y, y_dtype=F32)
    check(y, want, LINEAR_TOL, "y over its residual, strided rows")
    assert torch.equal(yw[:, 90:], rest)
    one = gdn.gdn_linear(x[:1].expand(M, 256), w, y_dtype=F32)
    assert torch.equal(one, one[:1].expand(M, 90))


def test_linear_non_finite_rows_stay_apart():
    x = torch.randn(70, 128, device="cuda").to(BF16)
    w = torch.randn(80, 128, device="cuda").to(BF16)
    y1 = gdn.gdn_linear(x, w)
    x[17, 3], w[33, 5] = float("nan"), float("inf")
    y2 = gdn.gdn_linear(x, w)
    assert torch.isnan(y2[17]).all() and not torch.isfinite(y2[:, 33]).any()
    keep = torch.ones_like(y1, dtype=torch.bool)
    keep[17], keep[:, 33] = False, False
    assert torch.equal(y1[keep], y2[keep])


# ----------------------------------------------------------------------------
# refusals of the binding
# ----------------------------------------------------------------------------

def test_refusals():
    d = make(10)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    cu = i32(0, 10)
    with pytest.raises(TypeError):
        gdn.gdn_prefill(d["q"].half(), *args[1:], cu, d["S"])
    with pytest.raises(TypeError):
        gdn.gdn_prefill(d["q"], d["k"].float(), *args[2:], cu, d["S"])
    with pytest.raises(ValueError):
        gdn.gdn_prefill(d["q"].cpu(), *args[1:], cu, d["S"])
    with pytest.raises(ValueError):
        gdn.gdn_prefill(*args[:3], d["g"][:5], d["beta"], cu, d["S"])
    with pytest.raises(ValueError):  # elements of a token are not dense
        gdn.gdn_prefill(d["q"].transpose(0, 1).contiguous().transpose(0, 1), *args[1:], cu, d["S"])
    with pytest.raises(gdn.GdnError, match="n_slots"):
        gdn.gdn_prefill(*args, i32(0, 5, 10), d["S"])
    with pytest.raises(gdn.GdnError, match="WORKSPACE"):
        gdn.gdn_prefill(*args, cu, d["S"], workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gdn.GdnError, match="ALIGN"):
        shifted = torch.zeros(41, device="cuda")[1:].view(10, 4)  # 4 bytes off a 16-byte boundary
        gdn.gdn_decode(*args[:3], shifted, d["beta"], d["S"].expand(10, 4, 128, 128).contiguous())
    with pytest.raises(ValueError):
        gdn.gdn_gated_norm(d["v"], d["v"], torch.ones(128, device="cuda"), gate="gelu")
    with pytest.raises(gdn.GdnError, match="SHAPE"):
        gdn.gdn_add_norm(torch.zeros(2, 16392, device="cuda"), None, torch.ones(16392, device="cuda"))
    x = torch.zeros(4, 8, dtype=BF16, device="cuda")
    with pytest.raises(ValueError):
        gdn.gdn_linear(x, x, act="relu")
    with pytest.raises(ValueError):
        gdn.gdn_linear(x, torch.zeros(4, 9, dtype=BF16, device="cuda"))
    with pytest.raises(TypeError):
        gdn.gdn_linear(x.float(), x)
