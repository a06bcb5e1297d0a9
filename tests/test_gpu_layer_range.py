"""gdn_prefill over the range that the header states and at its edge, |k|^2 =
2 with beta = 1 and no decay, against the recurrence in 64 bits.

Tolerances, in rel-L2.  Every fp32 operand of the chunked path's products is
held in three bf16 parts (24 bits), so its arithmetic is that of fp32:
 - typical gates forget, so an error is some 30 roundings of 2^-24: 2e-6, as
   for the token by token path;
 - at the edge nothing is forgotten: every token reflects the state, and the
   roundings of n tokens add, at random signs sqrt(n) of a few 2^-24 each.
   n = 2048: 45 * 5 * 2^-24 = 1.4e-5, within 2^-16 = 1.5e-5.
"""
import pytest

torch = pytest.importorskip("torch")
gdn = pytest.importorskip("gated_deltanet_tree_gdn_amd")

from test_gpu_layer import BF16, CHUNK_TOL, F32, FP32_TOL, check, gpu, i32, make, recurrence, say  # noqa: E402,F401

pytestmark = pytest.mark.gpu


def run(d, tol, what):
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    n, S = d["q"].shape[0], d["S"].clone()
    o = gdn.gdn_prefill(*args, i32(0, n), S, o_dtype=F32)
    want, end = recurrence(*args, d["S"][0])
    check(o, want, tol, f"{what}: o")
    check(S[0], end, tol, f"{what}: S")


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("rate", [0.01, 0.2])
@pytest.mark.parametrize("n", [70, 2000])
def test_fp32_outputs_of_typical_inputs(n, rate, dk, dv):
    say(f"[prefill] {n} tokens, decays of up to {2 * rate}, d {dk} {dv}")
    run(make(n, 1, 2, dk, dv, seed=n, rate=rate), FP32_TOL, f"{n} tokens")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dims", [2, 8, 128])
def test_keys_at_the_edge_of_the_range(dims, dtype):
    """|k|^2 just below 2, in few dimensions too: keys that nearly repeat"""
    say(f"[prefill] keys in {dims} dimensions, {dtype}")
    d = make(2048, 1, 2, seed=dims, dtype=F32)
    k = d["k"].clone()
    k[..., dims:] = 0
    k = k / k.norm(dim=-1, keepdim=True) * (2.0 * (1 - 2.0 ** -7)) ** 0.5  # below 2 after rounding too
    d = {a: (x.to(dtype) if a in ("q", "v") else x) for a, x in d.items()}
    d["k"] = k.to(dtype)
    assert d["k"].float().square().sum(-1).max() <= 2.0
    d["beta"].fill_(1.0)
    d["g"].zero_()
    run(d, CHUNK_TOL, f"{dims} dimensions")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("name", ["k", "q"])
@pytest.mark.parametrize("at", [0, 20, 40, 63, 100])
def test_zero_vectors_without_an_epsilon_stay_behind(at, name, dtype):
    """0 / 0: no earlier token and no other key head sees it; a key reaches every later token, a query its own"""
    d = make(130, 2, 4, seed=at, dtype=dtype)
    args = [d[a] for a in ("q", "k", "v", "g", "beta")]
    runs = []
    for i in range(2):
        S = d["S"].clone()
        o = gdn.gdn_prefill(*args, i32(0, 130), S, qk_l2norm=True, l2_eps=0.0, o_dtype=F32)
        runs.append((o, S))
        d[name][at, 1] = 0.0
    (o1, S1), (o2, S2) = runs
    assert torch.isfinite(o1).all() and torch.isfinite(S1).all()
    check(o2[:at], o1[:at], FP32_TOL, "tokens before it")
    check(o2[:, :2], o1[:, :2], FP32_TOL, "the other key head")
    check(S2[0, :2], S1[0, :2], FP32_TOL, "the other key head's state")
    if name == "k":
        assert torch.isnan(o2[at:, 2:]).all() and torch.isnan(S2[0, 2:]).all()
    else:
        assert torch.isnan(o2[at, 2:]).all()
        check(o2[at + 1:], o1[at + 1:], FP32_TOL, "later tokens")
        check(S2, S1, FP32_TOL, "S")


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("n", [1, 9, 449, 1500])
def test_the_walk_in_fp32(n, dk, dv):
    """q, k and v in fp32 are walked token by token at any length: the bound of that path, not of the chunks"""
    run(make(n, 1, 2, dk, dv, seed=n, dtype=F32), FP32_TOL, f"{n} tokens")
