"""gdn_prefill with offsets that are not in order: a bad entry makes its own
two sequences empty and leaves every other one right, whatever the workspace
held.  Tolerances as for the other tests of these operators."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from test_gpu_layer import BF16, CHUNK_TOL, F32, check, gpu, i32, make, recurrence, say  # noqa: E402,F401

pytestmark = pytest.mark.gpu

MANY = [0]  # 130 sequences, each 64 th entry out of range
for _b in range(130):
    MANY.append(MANY[-1] + (3 * _b) % 25)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cu", [
    [0, 500, -1, 600],       # a slot of the first sequence would be looked up as the third's
    [0, 190, -1, 199],
    [0, 200, 100, 300],      # two that overlap
    [0, 640, 64, 700],
    [-3, 70, 200, 150, 300, 900, 300, 301],
    [300, 0, 300],
    [2000000000, 0, 200, -2000000000, 200, 300],
    [x if b % 64 != 63 else [-1, 1 << 30][b // 64 % 2] for b, x in enumerate(MANY)],
], ids=lambda cu: str(cu[:6]))
@pytest.mark.parametrize("dk,dv", [(128, 64), (64, 128)])
def test_bad_offsets_leave_the_others_right(cu, dtype, dk, dv):
    T, B = max([x for x in cu if x <= 1000], default=0), len(cu) - 1
    T = min(T, 700)
    T += 8 * B + 1 if T <= 8 * B else 0  # enough tokens for chunks
    say(f"[prefill] T {T}, offsets {cu[:8]}, {dtype}")
    d = make(T, 1, 2, dk, dv, dtype=dtype, slots=B, seed=T)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    good = [b for b in range(B) if 0 <= cu[b] <= cu[b + 1] <= T]
    has = [b % 3 != 1 for b in range(B)]
    owners = torch.zeros(T, dtype=torch.int32)
    for b in good:
        owners[cu[b]:cu[b + 1]] += 1
    want_o, want_S = torch.full(d["v"].shape, 7.0, dtype=torch.double), d["S"].cpu().double()
    for b in range(B):
        start = d["S"][b] if has[b] else torch.zeros_like(d["S"][b])
        x = slice(cu[b], cu[b + 1]) if b in good else slice(0, 0)
        want_o[x], want_S[b] = recurrence(*(a[x] for a in args), start, 0.5, True)
    need = gdn.gdn_prefill_workspace_bytes(d["q"], d["v"], i32(*cu))
    for fill in (0, 255):
        S, status = d["S"].clone(), torch.full((B,), 77, dtype=torch.int32, device="cuda")
        o = torch.full(d["v"].shape, 7.0, device="cuda")
        gdn.gdn_prefill(*args, i32(*cu), S, has_state=i32(*map(int, has)), o=o, seq_status=status, q_scale=0.5,
                        qk_l2norm=True, workspace=torch.full((max(need, 1),), fill, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert status.tolist() == [0 if b in good else 2 for b in range(B)]
        one = (owners == 1).nonzero()[:, 0]
        if len(one):
            check(o[one.cuda()], want_o[one], CHUNK_TOL, "o of tokens with one owner")
        assert (o[(owners == 0).cuda()] == 7.0).all()
        for b in range(B):
            check(S[b], want_S[b], CHUNK_TOL, f"S of sequence {b}")
