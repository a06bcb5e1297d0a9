"""The Gated DeltaNet layer's operators as measured cases: the delta rule over
prompts and over single tokens, the norms around the layer, and its
projections.

``run`` computes an operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end), or with ``own`` true through this
package's entry points.  ``exact`` computes the same outputs in 64 bits from
each operator's definition, apart from the plain form.
"""
import math

import torch

own = False

C = 64  # tokens of one chunk of the plain form

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one long prompt on an idle GPU: 32 value heads are all the parallelism there is
        dict(name="prefill_long", op="prefill", B=1, T=16384, Hk=16, Hv=32, dk=128, dv=128, dtype="bf16",
             o_dtype="bf16", l2norm=True, resume=0.0),
        # a prefill step of a serving loop: prompts of very different lengths packed, some resuming a state
        dict(name="prefill_packed", op="prefill", B=13, T=7919, Hk=16, Hv=32, dk=128, dv=128, dtype="bf16",
             o_dtype="bf16", l2norm=True, resume=0.5),
        # short prompts of a small layer in 32 bits, as a checker runs them
        dict(name="prefill_small_f32", op="prefill", B=5, T=301, Hk=4, Hv=8, dk=64, dv=64, dtype="f32",
             o_dtype="f32", l2norm=False, resume=0.5),
        # one user generating: latency
        dict(name="decode_one", op="decode", B=1, slots=4, Hk=16, Hv=32, dk=128, dv=128, dtype="bf16",
             o_dtype="bf16", l2norm=True, idle=0.0),
        # a full batch, some of its rows idle, states scattered over a pool
        dict(name="decode_batch", op="decode", B=120, slots=144, Hk=16, Hv=32, dk=128, dv=128, dtype="bf16",
             o_dtype="f32", l2norm=True, idle=0.05),
        # the norm before the layer for one token: latency
        dict(name="add_norm_token", op="add_norm", T=1, D=4096, x="bf16", res="bf16", post=False, chan=False),
        # a packed prompt step, norms on both sides of the block, an odd number of rows
        dict(name="add_norm_prompt", op="add_norm", T=8191, D=5120, x="bf16", res="f32", post=True, chan=True),
        # the gated norm after the layer for a verify of one small tree
        dict(name="gated_norm_tree", op="gated_norm", T=37, H=32, d=128, x="f32", gate="silu"),
        # the same for a long prompt
        dict(name="gated_norm_prompt", op="gated_norm", T=16384, H=32, d=128, x="bf16", gate="silu"),
        # the input projection (q, k, v, z and the two gates of every value head) of one token: reads the weights once
        dict(name="linear_token", op="linear", M=1, N=12352, K=4096, bias=True, act="none", residual="none", y="bf16"),
        # the output projection of a verify step, ragged rows, with the residual
        dict(name="linear_ragged", op="linear", M=777, N=4096, K=4096, bias=True, act="silu", residual="bf16", y="bf16"),
        # the input projection of a long prompt
        dict(name="linear_prompt", op="linear", M=16384, N=12352, K=4096, bias=False, act="none", residual="none",
             y="bf16"),
    ]


def _log(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = max(lo, min(hi, n))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["prefill", "prefill", "decode", "add_norm", "gated_norm", "linear", "linear"])
    if op == "prefill":
        Hk, r = rng.choice([2, 4, 8, 16]), rng.choice([1, 2, 2, 4])
        f32 = rng.random() < 0.25
        Hv = min(Hk * r, 32)
        T = _log(rng, 1, 1500 if f32 else 16384)
        return dict(op=op, B=_log(rng, 1, 32), T=T, Hk=Hk, Hv=Hv, dk=rng.choice([64, 128]), dv=rng.choice([64, 128]),
                    dtype="f32" if f32 else "bf16", o_dtype=rng.choice(["bf16", "f32"]), l2norm=rng.random() < 0.5,
                    resume=rng.choice([0.0, 0.5, 1.0]))
    if op == "decode":
        Hk, r = rng.choice([2, 4, 8, 16]), rng.choice([1, 2, 2, 4])
        B = _log(rng, 1, 120)
        return dict(op=op, B=B, slots=B + rng.randint(0, 24), Hk=Hk, Hv=min(Hk * r, 32), dk=rng.choice([64, 128]),
                    dv=rng.choice([64, 128]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    o_dtype=rng.choice(["bf16", "f32"]), l2norm=rng.random() < 0.5, idle=rng.choice([0.0, 0.2]))
    if op == "add_norm":
        D = _log(rng, 60, 8200)
        return dict(op=op, T=_log(rng, 1, 8191 * 5120 // max(D, 5120)), D=D, x=rng.choice(["bf16", "f32"]),
                    res=rng.choice(["bf16", "f32"]), post=rng.random() < 0.5, chan=rng.random() < 0.3)
    if op == "gated_norm":
        return dict(op=op, T=_log(rng, 1, 16384), H=rng.choice([1, 4, 7, 16, 32]), d=rng.choice([64, 80, 128, 33]),
                    x=rng.choice(["bf16", "f32"]), gate=rng.choice(["silu", "sigmoid"]))
    K = _log(rng, 64, 4096)
    if rng.random() < 0.75:
        K = max(64, K // 64 * 64)
    return dict(op=op, M=_log(rng, 1, 16384), N=_log(rng, 16, 12352), K=K, bias=rng.random() < 0.5,
                act=rng.choice(["none", "silu", "gelu", "sigmoid"]), residual=rng.choice(["none", "bf16", "f32"]),
                y=rng.choice(["bf16", "f32"]))


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _lengths(B, T, seed):
    """B lengths that sum to T, spread over two orders of magnitude (some may be zero)."""
    g = torch.Generator().manual_seed(seed * 7919 + 11)
    w = torch.exp(2.3 * (2 * torch.rand(B, generator=g) - 1)).double()
    cut = torch.cat([torch.zeros(1, dtype=torch.double), torch.cumsum(w / w.sum(), 0)]) * T
    cu = cut.round().to(torch.int64)
    cu[-1] = T
    return cu


def _gates(n, Hv, gen):
    """Log-decays with a rate of each head's own, from almost none to strong, and write strengths in (0, 1)."""
    dev = "cuda"
    rate = torch.exp(torch.linspace(math.log(0.005), math.log(2.0), Hv, device=dev))
    g = -rate * torch.nn.functional.softplus(torch.randn(n, Hv, generator=gen, device=dev))
    beta = torch.sigmoid(torch.randn(n, Hv, generator=gen, device=dev))
    return g, beta


def _qkv(n, c, gen):
    """q, k and v as slices of one projection's rows; without the L2 norm in the operator, q and k come normalised."""
    Hk, Hv, dk, dv = c["Hk"], c["Hv"], c["dk"], c["dv"]
    dt = DTYPES[c["dtype"]]
    if c["l2norm"]:
        rows = torch.randn(n, 2 * Hk * dk + Hv * dv, generator=gen, device="cuda").to(dt)
        q, k, v = rows.split([Hk * dk, Hk * dk, Hv * dv], dim=1)
        return q.unflatten(1, (Hk, dk)), k.unflatten(1, (Hk, dk)), v.unflatten(1, (Hv, dv))
    q, k = (torch.randn(n, Hk, dk, generator=gen, device="cuda") for _ in range(2))
    q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
    return q.to(dt), k.to(dt), torch.randn(n, Hv, dv, generator=gen, device="cuda").to(dt)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    s = {"case": c}
    randn = lambda *n: torch.randn(*n, generator=gen, device="cuda")  # noqa: E731
    if c["op"] in ("prefill", "decode"):
        n = c["T"] if c["op"] == "prefill" else c["B"]
        s["q"], s["k"], s["v"] = _qkv(n, c, gen)
        s["g"], s["beta"] = _gates(n, c["Hv"], gen)
        slots = c["B"] if c["op"] == "prefill" else c["slots"]
        s["S"] = 0.5 * randn(slots, c["Hv"], c["dv"], c["dk"])
        s["q_scale"] = c["dk"] ** -0.5
    if c["op"] == "prefill":
        cu = _lengths(c["B"], c["T"], seed)
        s["lengths"] = (cu[1:] - cu[:-1]).tolist()
        s["cu"] = cu.to(torch.int32).cuda()
        s["has"] = (torch.rand(c["B"], generator=cpu) < c["resume"]).to(torch.int32).cuda()
        s["slot"] = torch.randperm(c["B"], generator=cpu).to(torch.int32).cuda()
    elif c["op"] == "decode":
        slot = torch.randperm(c["slots"], generator=cpu)[: c["B"]]
        slot[torch.rand(c["B"], generator=cpu) < c["idle"]] = -1
        s["slot"] = slot.to(torch.int32).cuda()
    elif c["op"] == "add_norm":
        s["x"] = randn(c["T"], c["D"]).to(DTYPES[c["x"]])
        s["res"] = (3.0 * randn(c["T"], c["D"])).to(DTYPES[c["res"]])
        s["w"] = 1.0 + 0.1 * randn(c["D"])
        s["post"] = 1.0 + 0.1 * randn(c["D"]) if c["post"] else None
        s["chan"] = 0.5 + 0.1 * randn(c["D"]) if c["chan"] else None
        s["scale"] = 0.7
    elif c["op"] == "gated_norm":
        T, H, d = c["T"], c["H"], c["d"]
        s["o"] = (0.3 * randn(T, H, d)).to(DTYPES[c["x"]])
        rows = randn(T, 2 * H * d).to(torch.bfloat16)  # the gate is a slice of a wider projection
        s["z"] = rows[:, H * d:].unflatten(1, (H, d))
        s["w"] = 1.0 + 0.1 * randn(d)
    elif c["op"] == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        s["x"] = randn(M, K).to(torch.bfloat16)
        s["w"] = (randn(N, K) * K ** -0.5).to(torch.bfloat16)
        s["bias"] = 0.1 * randn(N) if c["bias"] else None
        s["res"] = randn(M, N).to(DTYPES[c["residual"]]) if c["residual"] != "none" else None
        s["scale"] = 0.7 if s["res"] is not None else 1.0
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _heads(x, Hv):
    """Value head h reads key head h // (Hv / Hk)."""
    return x.repeat_interleave(Hv // x.shape[-2], dim=-2)


def _unit(x, l2norm):
    x = x.float()
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS) if l2norm else x


def _plain_prefill(s):
    """The delta rule in chunks of C tokens, every sequence padded to the longest."""
    c = s["case"]
    B, Hv, dv = c["B"], c["Hv"], c["dv"]
    cu = s["cu"].long()
    longest = max(s["lengths"])
    n = max(1, -(-longest // C))
    at = cu[:-1, None] + torch.arange(n * C, device="cuda")
    real = at < cu[1:, None]
    at = torch.where(real, at, 0)

    def chunks(x):  # [T][Hv][...] -> [B][Hv][n][C][...], zero where a sequence has ended
        x = torch.where(real.view(B, n * C, *[1] * (x.dim() - 1)), x[at], 0.0)
        return x.unflatten(1, (n, C)).movedim(3, 1)

    q = chunks(_heads(_unit(s["q"], c["l2norm"]) * s["q_scale"], Hv))
    k = chunks(_heads(_unit(s["k"], c["l2norm"]), Hv))
    v, beta = chunks(s["v"].float()), chunks(s["beta"])
    G = chunks(s["g"]).cumsum(-1)
    i = torch.arange(C, device="cuda")
    low = i[:, None] >= i
    D = torch.where(low, torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], 0.0)), 0.0)
    A = beta[..., None] * D * (k @ k.transpose(-1, -2)) * (i[:, None] > i)
    inv = torch.eye(C, device="cuda").expand_as(A).clone()  # (I + A)^-1 by forward substitution
    for r in range(1, C):
        inv[..., r, :r] = -(A[..., r, None, :r] @ inv[..., :r, :r])[..., 0, :]
    M = D * (q @ k.transpose(-1, -2))
    gamma, last = torch.exp(G)[..., None], torch.exp(G[..., -1:] - G)[..., None]
    slot = s["slot"].long()
    S = torch.where(s["has"].bool()[:, None, None, None], s["S"][slot], 0.0)
    o = torch.empty(B, Hv, n, C, dv, device="cuda")
    for j in range(n):
        St = S.transpose(-1, -2)
        u = inv[:, :, j] @ (beta[:, :, j, :, None] * (v[:, :, j] - gamma[:, :, j] * (k[:, :, j] @ St)))
        o[:, :, j] = gamma[:, :, j] * (q[:, :, j] @ St) + M[:, :, j] @ u
        S = gamma[:, :, j, -1:] * S + (last[:, :, j] * u).transpose(-1, -2) @ k[:, :, j]
    s["S"][slot] = S
    return o.movedim(1, 3).flatten(1, 2)[real].to(DTYPES[c["o_dtype"]]), s["S"]


def _plain_decode(s):
    c = s["case"]
    live = s["slot"] >= 0
    slot = s["slot"].long().clamp(min=0)
    q = _heads(_unit(s["q"], c["l2norm"]) * s["q_scale"], c["Hv"])[..., None, :]
    k = _heads(_unit(s["k"], c["l2norm"]), c["Hv"])[..., None, :]
    S = s["S"][slot] * torch.exp(s["g"])[..., None, None]
    u = s["beta"][..., None] * (s["v"].float() - (S * k).sum(-1))
    S = S + u[..., None] * k
    o = (S * q).sum(-1) * live[:, None, None]
    s["S"][slot[live]] = S[live]
    return o.to(DTYPES[c["o_dtype"]]), s["S"]


def _rms(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain_add_norm(s):
    x = s["x"].float()
    if s["post"] is not None:
        x = _rms(x) * s["post"]
    if s["chan"] is not None:
        x = x * s["chan"]
    h = s["res"].float() + s["scale"] * x
    return (_rms(h) * s["w"]).bfloat16(), h.to(s["res"].dtype)


def _plain_gated_norm(s):
    z = s["z"].float()
    gate = 1.0 / (1.0 + torch.exp(-z))
    if s["case"]["gate"] == "silu":
        gate = z * gate
    return (_rms(s["o"].float()) * s["w"] * gate).bfloat16()


def _plain_linear(s):
    c = s["case"]
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * 0.5 ** 0.5))
    elif c["act"] != "none":
        y = (y if c["act"] == "silu" else 1.0) / (1.0 + torch.exp(-y))
    if s["res"] is not None:
        y = s["res"].float() + s["scale"] * y
    return y.to(DTYPES[c["y"]])


def _own(s):
    import gated_deltanet_tree_gdn_amd as gdn
    c = s["case"]
    if c["op"] == "prefill":
        o = gdn.gdn_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], s["S"], slot=s["slot"],
                            has_state=s["has"], q_scale=s["q_scale"], qk_l2norm=c["l2norm"], l2_eps=EPS,
                            o_dtype=DTYPES[c["o_dtype"]])
        return o, s["S"]
    if c["op"] == "decode":
        o = gdn.gdn_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["S"], slot=s["slot"], q_scale=s["q_scale"],
                           qk_l2norm=c["l2norm"], l2_eps=EPS, o_dtype=DTYPES[c["o_dtype"]])
        return o, s["S"]
    if c["op"] == "add_norm":
        return gdn.gdn_add_norm(s["x"], s["res"], s["w"], scale=s["scale"], chan_scale=s["chan"],
                                post_weight=s["post"], eps=EPS)
    if c["op"] == "gated_norm":
        return gdn.gdn_gated_norm(s["o"], s["z"], s["w"], eps=EPS, gate=c["gate"])
    return gdn.gdn_linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["res"], scale=s["scale"],
                          y_dtype=DTYPES[c["y"]])


def run(state):
    if own:
        return _own(state)
    return {"prefill": _plain_prefill, "decode": _plain_decode, "add_norm": _plain_add_norm,
            "gated_norm": _plain_gated_norm, "linear": _plain_linear}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without, and its outputs in 64 bits
# ----------------------------------------------------------------------------

def work(case):
    c, size = case, {"bf16": 2, "f32": 4, "none": 0}
    if c["op"] in ("prefill", "decode"):
        n = c["T"] if c["op"] == "prefill" else c["B"] * (1 - c["idle"])
        read = c["B"] * c["resume"] if c["op"] == "prefill" else n  # states read; every sequence's is written
        written = c["B"] if c["op"] == "prefill" else n
        state = 4 * c["Hv"] * c["dk"] * c["dv"]
        token = (size[c["dtype"]] * (2 * c["Hk"] * c["dk"] + c["Hv"] * c["dv"]) + 8 * c["Hv"]
                 + size[c["o_dtype"]] * c["Hv"] * c["dv"])
        return {"bytes": n * token + (read + written) * state, "flops": 6 * n * c["Hv"] * c["dk"] * c["dv"]}
    if c["op"] == "add_norm":
        n = c["T"] * c["D"]
        return {"bytes": n * (size[c["x"]] + 2 * size[c["res"]] + 2) + 4 * c["D"] * (1 + c["post"] + c["chan"]),
                "flops": n * (8 if c["post"] else 5)}
    if c["op"] == "gated_norm":
        n = c["T"] * c["H"] * c["d"]
        return {"bytes": n * (size[c["x"]] + 4) + 4 * c["d"], "flops": 8 * n}
    M, N, K = c["M"], c["N"], c["K"]
    return {"bytes": 2 * (M + N) * K + M * N * (size[c["y"]] + size[c["residual"]]) + 4 * N * c["bias"],
            "flops": 2 * M * N * K}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    d = lambda x: None if x is None else x.double()  # noqa: E731
    if c["op"] in ("prefill", "decode"):
        q, k, v, g, beta, S = (d(s[n]) for n in ("q", "k", "v", "g", "beta", "S"))
        if c["l2norm"]:
            q, k = (x / (x.pow(2).sum(-1, keepdim=True) + EPS).sqrt() for x in (q, k))
        group = c["Hv"] // c["Hk"]
        own_head = torch.arange(c["Hv"], device="cuda") // group
        q, k, alpha = (q * s["q_scale"])[:, own_head], k[:, own_head], g.exp()
        o = torch.zeros(v.shape, dtype=torch.double, device="cuda")

        def step(state, t):  # the definition: S <- a S (I - b k k^T) + b v k^T, then o = S q
            state = alpha[t, :, None, None] * state
            kt = k[t, :, :, None]
            state = state + (beta[t, :, None] * (v[t] - (state @ kt)[..., 0]))[..., None] * kt.transpose(-1, -2)
            o[t] = (state @ q[t, :, :, None])[..., 0]
            return state

        slot = s["slot"].tolist()
        if c["op"] == "decode":
            for b, at in enumerate(slot):
                if at >= 0:
                    S[at] = step(S[at], b)
        else:
            t, has = 0, s["has"].tolist()
            for b, length in enumerate(s["lengths"]):
                state = S[slot[b]] if has[b] else torch.zeros_like(S[slot[b]])
                for t in range(t, t + length):
                    state = step(state, t)
                t += 1 if length else 0
                S[slot[b]] = state
        return o, S
    if c["op"] == "add_norm":
        x = d(s["x"])
        if c["post"]:
            x = x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * d(s["post"])
        h = d(s["res"]) + s["scale"] * (x * d(s["chan"]) if c["chan"] else x)
        return h / (h.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * d(s["w"]), h
    if c["op"] == "gated_norm":
        o, z = d(s["o"]), d(s["z"])
        act = torch.sigmoid(z) * (z if c["gate"] == "silu" else 1.0)
        return o / (o.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * d(s["w"]) * act
    w = d(s["w"]).t().contiguous()
    y = torch.cat([d(x) @ w for x in s["x"].split(2048)])
    y = y if s["bias"] is None else y + d(s["bias"])
    if c["act"] == "gelu":
        y = y * 0.5 * (1 + torch.special.erf(y / math.sqrt(2.0)))
    elif c["act"] != "none":
        y = torch.sigmoid(y) * (y if c["act"] == "silu" else 1.0)
    return y if s["res"] is None else d(s["res"]) + s["scale"] * y
