"""What the Python binding of gdn_layer.h checks and allocates."""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from test_gpu_layer import BF16, F32, gpu, i32, make  # noqa: E402,F401

pytestmark = pytest.mark.gpu

WORKSPACES = [  # none of these is memory that a kernel may write to
    (lambda n: torch.empty(n, dtype=torch.uint8), ValueError),
    (lambda n: torch.empty(1, dtype=torch.uint8, device="cuda").expand(n), ValueError),
    (lambda n: torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2], ValueError),
    (lambda n: torch.empty(n, device="cuda"), TypeError),
    (lambda n: bytearray(n), TypeError),
]


@pytest.mark.parametrize("make_ws,error", WORKSPACES)
def test_a_workspace_is_checked(make_ws, error):
    d = make(200)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    cu = i32(0, 200)
    need = gdn.gdn_prefill_workspace_bytes(d["q"], d["v"], cu)
    assert need > 0
    with pytest.raises(error, match="workspace"):
        gdn.gdn_prefill(*args, cu, d["S"], workspace=make_ws(need))
    x, w = (torch.zeros(600, 129, dtype=BF16, device="cuda")[:, :128] for _ in range(2))  # rows that are copied first
    with pytest.raises(error, match="workspace"):
        gdn.gdn_linear(x, w, workspace=make_ws(1 << 20))
    y = gdn.gdn_linear(x, w, workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    assert (y == 0).all()


# one call of every operator whose output (or workspace) has `n` bytes
def calls(n, stream):
    T = n // (4 * 128 * 4)
    d = make(T, slots=T)
    v, w, cu = d["v"], torch.ones(128, device="cuda"), i32(0, T)
    rows = v.flatten(1)
    big = torch.zeros(T, 1030, dtype=BF16, device="cuda")[:, :1026]  # 1026 elements padded to 1032 when copied
    small = torch.zeros(1024, 1026, dtype=BF16, device="cuda")[:, :1026]
    qkv = [d[a] for a in ("q", "k", "v", "g", "beta")]
    f32 = [x.float() if i < 3 else x for i, x in enumerate(qkv)]
    out = torch.empty(T, 512, device="cuda")
    need = gdn.gdn_prefill_workspace_bytes(d["q"], v, cu)
    y = torch.empty(T, 1024, dtype=BF16, device="cuda")
    from gated_deltanet_tree_gdn_amd import layer
    copied = layer.layer_library().gdn_linear_workspace_bytes(
        layer.LinearDims(T, 1024, 1026, 0, 0, 0, 1.0, big.stride(0), small.stride(0), 0, 1024))
    assert need > 0 and copied > 0
    return {
        "prefill": (n, lambda: gdn.gdn_prefill(*f32, cu, d["S"], o_dtype=F32, stream=stream)),
        "prefill workspace": (need, lambda: gdn.gdn_prefill(*qkv, cu, d["S"], o=out.view(T, 4, 128), stream=stream)),
        "decode": (n, lambda: gdn.gdn_decode(*qkv, d["S"], o_dtype=F32, stream=stream)),
        "add_norm": (n, lambda: gdn.gdn_add_norm(rows, None, w.repeat(4), h=rows, y_dtype=F32, stream=stream)),
        "gated_norm": (n, lambda: gdn.gdn_gated_norm(v, v, w, y_dtype=F32, stream=stream)),
        "linear": (2 * n, lambda: gdn.gdn_linear(rows, rows[:1024].contiguous(), y_dtype=F32, stream=stream)),
        "linear workspace": (copied, lambda: gdn.gdn_linear(big, small, y=y, stream=stream)),
    }


NAMES = ["prefill", "prefill workspace", "decode", "add_norm", "gated_norm", "linear", "linear workspace"]


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_reads_is_not_taken(name, raw):
    """a freed block waits for its stream: a call on another stream must not get it before then"""
    side = torch.cuda.Stream()
    size, call = calls(4 << 20, side.cuda_stream if raw else side)[name]
    call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    kept = torch.empty(size, dtype=torch.uint8, device="cuda")
    old = torch.full((size,), 77, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(200_000_000)  # some 0.1 s
    kept.copy_(old)
    del old
    out = call()
    torch.cuda.synchronize()
    assert (kept == 77).all(), name
    del out


def test_outputs_of_another_stream_outlive_their_use_on_this_one():
    side = torch.cuda.Stream()
    size, call = calls(4 << 20, side)["gated_norm"]
    y = call()
    want = y.clone()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    kept = torch.empty_like(y)
    want.copy_(y)
    torch.cuda._sleep(200_000_000)
    kept.copy_(y)
    del y
    with torch.cuda.stream(side):
        junk = [torch.full((size // 4,), 3.0, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and len(junk) == 4


def test_a_call_on_the_default_stream_from_another():
    d = make(300)
    w = torch.ones(128, device="cuda")
    want = gdn.gdn_gated_norm(d["v"], d["v"], w)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for s in (0, torch.cuda.default_stream()):
            y = gdn.gdn_gated_norm(d["v"], d["v"], w, stream=s)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
