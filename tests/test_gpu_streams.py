"""Outputs that the binding of gdn_tree.h allocates for a call on another
stream than the current one: their memory must not be a block that the
current stream's earlier work still uses, nor be cleared behind the call."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from test_gpu_layer import gpu, make  # noqa: E402,F401

pytestmark = pytest.mark.gpu

B, N, NBYTES = 32, 64, 32 * 64 * 4 * 128 * 4


def setup():
    d = make(B * N, slots=B)
    args = [d[a].unflatten(0, (B, N)) for a in ("q", "k", "v", "g", "beta")]
    parent = ((torch.arange(N, device="cuda", dtype=torch.int32) - 1) // 2).repeat(B, 1).contiguous()
    parent[:, 0] = -1
    return args, parent, d["S"]


@pytest.mark.parametrize("name", ["verify", "branches", "static", "commit", "commit_verify"])
def test_memory_that_the_current_stream_still_reads_is_not_taken(name):
    args, parent, S0 = setup()
    side = torch.cuda.Stream()
    ctx = gdn.GdnContext.for_tensors(args[0], args[2], parent)
    accepted = torch.full((B,), N - 1, dtype=torch.int32, device="cuda")
    o = torch.empty(B, N, 4, 128, device="cuda")
    S_next = torch.empty_like(S0)
    gdn.gdn_tree_verify(ctx, *args, parent, S0, o=o)
    size, call = {
        "verify": (NBYTES, lambda s: gdn.gdn_tree_verify(ctx, *args, parent, S0, stream=s)),
        "branches": (NBYTES, lambda s: gdn.gdn_tree_verify_branches(ctx, *args, parent, S0, stream=s)),
        "static": (NBYTES, lambda s: gdn.gdn_tree_verify_static(*args, parent, S0, stream=s)),
        "commit": (S0.numel() * 4, lambda s: gdn.gdn_commit_path(ctx, accepted, stream=s)),
        "commit_verify": (NBYTES, lambda s: gdn.gdn_commit_verify(ctx, accepted, *args, parent, S_next=S_next, stream=s)[0]),
    }[name]
    want = call(None).clone()
    if name == "commit_verify":
        gdn.gdn_tree_verify(ctx, *args, parent, S0, o=o)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = torch.empty(size, dtype=torch.uint8, device="cuda")
    old = torch.full((size,), 77, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(200_000_000)  # some 0.1 s
    kept.copy_(old)
    del old
    got = call(side)
    torch.cuda.synchronize()
    assert (kept == 77).all() and torch.equal(got, want)


def test_ancestors_are_not_cleared_behind_the_call():
    _, parent, _ = setup()
    want = gdn.gdn_tree_ancestors(parent)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    got = gdn.gdn_tree_ancestors(parent, stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and want[0].any()
