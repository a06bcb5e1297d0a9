"""The attention layers between Gated DeltaNet layers as measured cases: keys
and values appended to a paged cache with norm and rotation, attention of
single tokens, of whole proposal trees and of packed prompts over that cache,
and the commit of a tree's accepted path in it.

``run`` computes an operator in its plain form (elementary torch operations
in 32 bits, rounded once at the end), or with ``own`` true through this
package's entry points.  ``exact`` computes the same outputs in 64 bits from
each operator's definition, apart from the plain form.
"""
import math
import random

import torch

own = False

EPS = 1e-6
THETA = 1e6
E4M3_MAX = 448.0
CACHE = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one user generating: the new token's query and key normed and rotated, key and value stored; latency
        dict(name="append_token", op="append", T=1, Hq=16, Hkv=2, d=256, rot=64, pairs="halves", norm=True, idle=0.0,
             cache="bf16", page=16),
        # a packed prompt step into an 8-bit cache, some rows of the batch being padding
        dict(name="append_prompt", op="append", T=12289, Hq=32, Hkv=8, d=128, rot=128, pairs="neighbours", norm=False,
             idle=0.03, cache="e4m3", page=64),
        # one user generating after a short chat: latency
        dict(name="decode_one", op="decode", B=1, total=1531, Hq=16, Hkv=2, d=256, gate=True, cache="bf16", page=16),
        # one user with a very long document: two key heads are all the parallelism there is beside the length
        dict(name="decode_long", op="decode", B=1, total=131071, Hq=16, Hkv=2, d=256, gate=True, cache="bf16", page=64),
        # a full batch of chats whose lengths differ by an order of magnitude
        dict(name="decode_batch", op="decode", B=96, total=400009, Hq=32, Hkv=8, d=128, gate=False, cache="bf16",
             page=16),
        # a batch of a smaller layer with six query heads to a key head and an 8-bit cache
        dict(name="decode_e4m3", op="decode", B=24, total=200003, Hq=24, Hkv=4, d=64, gate=False, cache="e4m3", page=32),
        # the verify of one small tree after a chat: latency
        dict(name="verify_tree", op="verify", B=1, N=48, total=2903, Hq=16, Hkv=2, d=256, gate=True, cache="bf16",
             page=16),
        # the verify of a batch of full trees
        dict(name="verify_batch", op="verify", B=16, N=128, total=100003, Hq=32, Hkv=8, d=128, gate=False, cache="bf16",
             page=16),
        # one long prompt
        dict(name="prefill_long", op="prefill", B=1, T=16384, cached=0, Hq=16, Hkv=2, d=256, gate=True, cache="bf16",
             page=64),
        # a prompt step of a serving loop: chunks of very different prompts, each behind what is cached of it
        dict(name="prefill_packed", op="prefill", B=9, T=6007, cached=20011, Hq=32, Hkv=8, d=128, gate=False,
             cache="e4m3", page=16),
        # the accepted path of one small tree, in the caches of all attention layers of a model
        dict(name="commit_one", op="commit", layers=12, B=1, N=48, path=5, total=803, Hkv=2, d=256, cache="bf16", page=16),
        # the same for a batch of full trees
        dict(name="commit_batch", op="commit", layers=12, B=32, N=128, path=8, total=12007, Hkv=2, d=256, cache="bf16",
             page=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_heads(rng):
    d = rng.choice([64, 128, 256])
    Hkv = rng.choice([1, 2, 3, 4, 8]) if d < 256 else rng.choice([1, 2, 4])
    return dict(Hq=Hkv * rng.choice([1, 2, 4, 6, 7, 8]), Hkv=Hkv, d=d)


def _pairs(c):
    """Query and key pairs that the mask of a prefill leaves, and those of the padded rectangle."""
    n, before = _lengths(c["T"], c["B"]), _lengths(c["cached"], c["B"])
    seen = sum(a * b + a * (a + 1) // 2 for a, b in zip(n, before))
    return seen, c["B"] * max(n) * max(a + b for a, b in zip(n, before))


def draw(rng):
    op = rng.choice(["append", "decode", "decode", "verify", "verify", "prefill", "prefill", "commit"])
    c = dict(op=op, **_draw_heads(rng), cache=rng.choice(["bf16", "bf16", "e4m3"]), page=rng.choice([8, 16, 32, 64, 128]))
    c["gate"] = rng.random() < 0.4
    row = c["Hkv"] * c["d"]
    if op == "append":
        del c["gate"]
        c.update(T=_log(rng, 1, 12289 * 40 * 128 // max(5120, (c["Hq"] + 2 * c["Hkv"]) * c["d"])),
                 rot=rng.choice([0, 32, 64, c["d"]]), pairs=rng.choice(["halves", "neighbours"]),
                 norm=rng.random() < 0.5, idle=rng.choice([0.0, 0.0, 0.1]))
    elif op == "decode":
        c.update(B=_log(rng, 1, 96))
        c.update(total=_log(rng, c["B"], min(400009, 400009 * 1024 // row, 131071 * c["B"])))
    elif op == "verify":
        c.update(B=_log(rng, 1, 16), N=_log(rng, 1, 200))
        c.update(total=_log(rng, c["B"], max(c["B"] + 1, min(100003, 100003 * 128 * 4096 // (c["N"] * c["Hq"] * c["d"])) // 2)))
    elif op == "prefill":
        c.update(B=_log(rng, 1, 16), T=_log(rng, 1, 16384), cached=rng.choice([0, _log(rng, 1, 30011)]))
        while _pairs(c)[1] * c["Hq"] > 16384 * 16384 * 10 or _pairs(c)[0] * c["Hq"] * c["d"] > 16384 * 8192 * 4096:
            c.update(T=(c["T"] + 1) // 2, cached=c["cached"] // 2)
    else:
        del c["gate"], c["Hq"]
        c.update(layers=rng.choice([1, 4, 12, 24]), B=_log(rng, 1, 32), N=_log(rng, 1, 200))
        c.update(path=rng.randint(0, min(c["N"], 12)))
        c.update(total=_log(rng, c["B"], 40000 * 512 // max(512, row) // c["layers"] + c["B"]))
    return c


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _lengths(total, B):
    """B lengths that sum to total, spread over more than an order of magnitude (some may be zero)."""
    rng = random.Random(total * 1009 + B)
    w = [math.exp(rng.uniform(-1.3, 1.3)) for _ in range(B)]
    ends = [round(total * sum(w[:b]) / sum(w)) for b in range(B + 1)]
    return [b - a for a, b in zip(ends, ends[1:])]


def _paged(c, lengths, gen, cpu):
    """The cache of a layer: pools of pages of keys and values, and the table of each sequence's pages, in no order."""
    page, counts = c["page"], [-(-n // c["page"]) for n in lengths]
    pool = sum(counts) + 5
    perm = torch.randperm(pool, generator=cpu).to(torch.int32)
    table = torch.full((len(lengths), max(max(counts), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = perm[at:at + n]
        at += n
    s = {"table": table.cuda(), "length": torch.tensor(lengths, dtype=torch.int32).cuda(), "most": max(lengths)}
    s["pool"], s["k_scale"], s["v_scale"] = pool, None, None
    if c["cache"] == "e4m3":
        s["k_scale"], s["v_scale"] = (x * torch.linspace(0.8, 1.2, c["Hkv"], device="cuda") for x in (0.02, 0.03))
    return s


def _pool(c, pool, gen, layers=None):
    """Keys or values of all pages (in 8 bits: as stored, to be multiplied by the scale of each head)."""
    shape = (pool, c["page"], c["Hkv"], c["d"])
    shape = shape if layers is None else (layers, *shape)
    if c["cache"] == "bf16":
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    return x.mul_(50.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _gate_rows(n, c, gen):
    """Query and gate of every head lie next to each other in the rows of one projection."""
    rows = torch.randn(n, c["Hq"], 2 * c["d"], generator=gen, device="cuda").to(torch.bfloat16)
    return rows[..., :c["d"]], rows[..., c["d"]:]


def _tree(N, path, cpu):
    """A random tree of N nodes as ancestor bits, and the node at the end of a root path of `path` nodes.  The path's
    first nodes are the first in the tree, as a best-first search finds them; the others lie behind the path's length."""
    lead = int(torch.randint(0, path + 1, (1,), generator=cpu)) if path else 0
    far = torch.randperm(max(N - path, 1), generator=cpu)[:path - lead].sort().values + path
    lead += path - lead - (far < N).sum().item() if N > path else path - lead
    nodes = (list(range(lead)) + far[far < N].tolist())[:path]
    parent = [int(torch.randint(-1, i, (1,), generator=cpu)) if i else -1 for i in range(N)]
    for before, node in zip([-1] + nodes, nodes):
        parent[node] = before
    up = []
    for i, p in enumerate(parent):
        up.append((up[p] if p >= 0 else 0) | 1 << i)
    words = [[((u >> 32 * w & 0xffffffff) ^ 0x80000000) - 0x80000000 for w in range((N + 31) // 32)] for u in up]
    return torch.tensor(words, dtype=torch.int32), nodes[-1] if nodes else -1


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    cpu = torch.Generator().manual_seed(seed)
    s = {"case": c}
    if c["op"] == "append":
        T, Hq, Hkv, d = c["T"], c["Hq"], c["Hkv"], c["d"]
        s.update(_paged(c, [T], gen, cpu))
        rows = torch.randn(T, (Hq + 2 * Hkv) * d, generator=gen, device="cuda").to(torch.bfloat16)
        s["q"], s["k_new"], s["v_new"] = (x.unflatten(1, (-1, d)) for x in rows.split([Hq * d, Hkv * d, Hkv * d], dim=1))
        at = torch.arange(T)
        slot = s["table"].cpu().long()[0, at // c["page"]] * c["page"] + at % c["page"]
        slot[torch.rand(T, generator=cpu) < c["idle"]] = -1
        s["slot"] = slot.to(torch.int32).cuda()
        s["position"] = (at + int(torch.randint(0, 131072, (1,), generator=cpu))).to(torch.int32).cuda()
        s["inv_freq"] = (THETA ** (-torch.arange(0, c["rot"], 2).double() / max(c["rot"], 1))).float().cuda()
        s["q_weight"], s["k_weight"] = (1.0 + 0.1 * torch.randn(d, generator=gen, device="cuda") if c["norm"] else None
                                        for _ in range(2))
        s["k"], s["v"] = (_pool(c, s["pool"], gen) for _ in range(2))
        return _with_handle(s)
    if c["op"] == "commit":
        order = torch.randperm(c["B"], generator=cpu).tolist()
        before = [_lengths(c["total"], c["B"])[b] for b in order]
        s.update(_paged(c, [n + c["N"] for n in before], gen, cpu))
        s["length"] = torch.tensor(before, dtype=torch.int32).cuda()
        trees = [_tree(c["N"], c["path"], cpu) for _ in before]
        s["anc"] = torch.stack([t[0] for t in trees]).cuda()
        s["accepted"] = torch.tensor([t[1] for t in trees], dtype=torch.int32).cuda()
        s["k"], s["v"] = (_pool(c, s["pool"], gen, c["layers"]) for _ in range(2))
        return _with_handle(s)
    order = torch.randperm(c["B"], generator=cpu).tolist()
    if c["op"] == "prefill":
        n, before = ([_lengths(x, c["B"])[b] for b in order] for x in (c["T"], c["cached"]))
        s["new"] = n
        s["cu"] = torch.tensor([sum(n[:b]) for b in range(c["B"] + 1)], dtype=torch.int32).cuda()
        lengths, rows = [a + b for a, b in zip(n, before)], c["T"]
    else:
        lengths = [_lengths(c["total"], c["B"])[b] for b in order]
        rows = c["B"] * c.get("N", 1)
    s.update(_paged(c, [n + c.get("N", 0) for n in lengths], gen, cpu))
    s["length"] = torch.tensor(lengths, dtype=torch.int32).cuda()
    s["k"], s["v"] = (_pool(c, s["pool"], gen) for _ in range(2))
    q, gate = _gate_rows(rows, c, gen)
    shape = (c["B"], c["N"]) if c["op"] == "verify" else (rows,)
    s["q"] = (2.0 * q).contiguous().unflatten(0, shape)  # as gdn_kv_append leaves it; scores spread by 2
    s["gate"] = gate.unflatten(0, shape) if c["gate"] else None
    if c["op"] == "verify":
        s["anc"] = torch.stack([_tree(c["N"], 0, cpu)[0] for _ in range(c["B"])]).cuda()
    return _with_handle(s)


def _with_handle(s):
    if own:
        import gated_deltanet_tree_gdn_amd as gdn
        if s["case"]["op"] == "commit":
            s["handle"] = [gdn.GdnKvCache(k, v, s["k_scale"], s["v_scale"]) for k, v in zip(s["k"], s["v"])]
        else:
            s["handle"] = gdn.GdnKvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return s


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------

def _plain_append(s):
    c = s["case"]
    q, k, v = s["q"].float(), s["k_new"].float(), s["v_new"].float()
    if c["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_weight"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_weight"]
    if c["rot"]:
        angle = s["position"].double()[:, None] * s["inv_freq"].double()
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
        half = c["rot"] // 2
        if c["pairs"] == "halves":
            first, second = slice(0, half), slice(half, c["rot"])
        else:
            first, second = slice(0, c["rot"], 2), slice(1, c["rot"], 2)
        turned = []
        for x in (q, k):
            y = x.clone()
            y[..., first] = x[..., first] * cos - x[..., second] * sin
            y[..., second] = x[..., second] * cos + x[..., first] * sin
            turned.append(y)
        q, k = turned
    live = s["slot"] >= 0
    slot = s["slot"][live].long()
    for pool, scale, x in ((s["k"], s["k_scale"], k), (s["v"], s["v_scale"], v)):
        if scale is not None:
            x = (x / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        pool[slot // c["page"], slot % c["page"]] = x[live].to(pool.dtype)
    return q.bfloat16(), s["k"], s["v"]


def _rows_of(s, name, keys):
    """The first `keys` cached rows of every sequence [B][H_kv][keys][d], in 32 bits."""
    x = s[name]
    x = x.view(torch.uint8)[s["table"].clamp(min=0).long()].view(x.dtype) if x.element_size() == 1 else \
        x[s["table"].clamp(min=0).long()]
    x = x.flatten(1, 2)[:, :keys].movedim(2, 1).float()
    scale = s[name + "_scale"]
    return x if scale is None else x * scale[:, None, None]


def _plain_attention(s, q, visible):
    """q [B][n][H_q][d] over the cached rows that visible [B][n][keys] leaves."""
    c = s["case"]
    B, n, G = q.shape[0], q.shape[1], c["Hq"] // c["Hkv"]
    q = q.float().unflatten(2, (c["Hkv"], G)).movedim(1, 3).flatten(2, 3)  # [B][H_kv][G n][d]
    k, v = (_rows_of(s, name, visible.shape[2]) for name in ("k", "v"))
    p = (q @ k.transpose(-1, -2)).mul_(c["d"] ** -0.5).unflatten(2, (G, n))
    p.masked_fill_(~visible[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (G, n)) / torch.where(total == 0, 1.0, total)
    return o.movedim(3, 1).flatten(2, 3)


def _gated(o, gate):
    return (o if gate is None else o / (1.0 + torch.exp(-gate.float()))).bfloat16()


def _plain_decode(s):
    visible = torch.arange(s["most"], device="cuda") < s["length"][:, None, None]
    return _gated(_plain_attention(s, s["q"][:, None], visible)[:, 0], s["gate"])


def _plain_verify(s):
    N = s["case"]["N"]
    behind = torch.arange(s["most"], device="cuda") - s["length"][:, None].long()  # node of a cached row, if any
    node = behind.clamp(0, N - 1)
    word = torch.gather(s["anc"], 2, (node // 32)[:, None].expand(-1, N, -1))
    bit = (word >> (node % 32).to(torch.int32)[:, None]) & 1
    visible = (behind < 0)[:, None] | ((behind < N)[:, None] & (bit != 0))
    return _gated(_plain_attention(s, s["q"], visible), s["gate"])


def _plain_prefill(s):
    cu = s["cu"].long()
    row = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.bucketize(row, cu[1:], right=True)
    at = row - cu[seq]
    q = s["q"].new_zeros(len(s["new"]), max(s["new"]), *s["q"].shape[1:])
    q[seq, at] = s["q"]
    new = cu[1:] - cu[:-1]
    last = (s["length"] - new)[:, None] + torch.arange(q.shape[1], device="cuda")
    visible = torch.arange(s["most"], device="cuda") <= last[..., None]
    return _gated(_plain_attention(s, q, visible)[seq, at], s["gate"])


def _plain_commit(s):
    c = s["case"]
    bits = s["anc"][torch.arange(c["B"], device="cuda"), s["accepted"].clamp(min=0).long()]  # [B][W]
    node = torch.arange(c["N"], device="cuda")
    on = ((bits[:, node // 32] >> (node % 32).to(torch.int32)) & 1).bool() & (s["accepted"] >= 0)[:, None]
    b, node = on.nonzero(as_tuple=True)
    to = s["length"][b] + on.cumsum(1)[b, node] - 1
    src = s["length"][b] + node

    def place(t):
        return s["table"][b, t // c["page"]].long(), t % c["page"]

    (from_page, from_row), (to_page, to_row) = place(src), place(to)
    for x in (s["k"], s["v"]):
        x = x.view(torch.uint8) if x.element_size() == 1 else x
        x[:, to_page, to_row] = x[:, from_page, from_row]
    return s["k"], s["v"], s["length"] + on.sum(1).to(torch.int32)


def _own(s):
    import gated_deltanet_tree_gdn_amd as gdn
    c, cache = s["case"], s["handle"]
    if c["op"] == "append":
        q = gdn.gdn_kv_append(cache, s["k_new"], s["v_new"], s["slot"], position=s["position"], inv_freq=s["inv_freq"],
                              q=s["q"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                              interleaved=c["pairs"] == "neighbours")
        return q, s["k"], s["v"]
    if c["op"] == "decode":
        return gdn.gdn_attn_decode(cache, s["q"], s["table"], s["length"], gate=s["gate"])
    if c["op"] == "verify":
        return gdn.gdn_attn_verify(cache, s["q"], s["anc"], s["table"], s["length"], gate=s["gate"])
    if c["op"] == "prefill":
        return gdn.gdn_attn_prefill(cache, s["q"], s["cu"], s["table"], s["length"], gate=s["gate"])
    length = gdn.gdn_kv_commit(cache, s["anc"], s["accepted"], s["table"], s["length"])
    return s["k"], s["v"], length


def run(state):
    if own:
        return _own(state)
    return {"append": _plain_append, "decode": _plain_decode, "verify": _plain_verify, "prefill": _plain_prefill,
            "commit": _plain_commit}[state["case"]["op"]](state)


# ----------------------------------------------------------------------------
# what a pass cannot do without, and its outputs in 64 bits
# ----------------------------------------------------------------------------

def work(case):
    c = case
    size = 2 if c["cache"] == "bf16" else 1
    row = 2 * size * c["Hkv"] * c["d"]  # a token's keys and values in the cache
    if c["op"] == "append":
        heads = c["Hq"] + c["Hkv"]
        return {"bytes": c["T"] * (2 * (2 * c["Hq"] + 2 * c["Hkv"]) * c["d"] + (1 - c["idle"]) * row + 8),
                "flops": c["T"] * (heads * (3 * c["rot"] + 4 * c["d"] * c["norm"]) + 8 * c["rot"])}
    if c["op"] == "commit":
        return {"bytes": c["layers"] * c["B"] * c["path"] * 2 * row + c["B"] * (c["N"] // 8 + 12), "flops": 0}
    if c["op"] == "prefill":
        rows, pairs, keys = c["T"], _pairs(c)[0], c["T"] + c["cached"]
    else:
        n = c.get("N", 1)
        rows, pairs = c["B"] * n, c["total"] * n + (c["B"] * n if c["op"] == "verify" else 0)
        keys = c["total"] + c["B"] * c.get("N", 0)
    return {"bytes": keys * row + rows * c["Hq"] * c["d"] * (4 + 2 * c["gate"]) + 4 * keys // c["page"],
            "flops": 4 * pairs * c["Hq"] * c["d"]}


def _exact_sequence(q, k, v, seen, scale):
    """Softmax attention of one sequence in 64 bits: q [n][H_q][d], k and v [keys][H_kv][d], seen(a, b) [b - a][keys]."""
    o = torch.zeros(q.shape, dtype=torch.double, device=q.device)
    group = q.shape[1] // k.shape[1]
    for h in range(q.shape[1]):
        kh, vh = k[:, h // group].double(), v[:, h // group].double()
        for a in range(0, q.shape[0], 4096):
            qh = q[a:a + 4096, h].double()
            z = (qh @ kh.t().contiguous()) * scale
            z[~seen(a, a + qh.shape[0])] = -math.inf
            some = (z > -math.inf).any(1)
            w = torch.softmax(z[some], dim=1)
            o[a:a + qh.shape[0], h][some] = w @ vh
    return o


def exact(case, seed):
    s, c = prepare(case, seed), case
    page = c["page"]
    if c["op"] == "append":
        q, k, v = s["q"].double(), s["k_new"].double(), s["v_new"].double()
        if c["norm"]:
            q, k = (x / (x.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s[w].double()
                    for x, w in ((q, "q_weight"), (k, "k_weight")))
        if c["rot"]:
            turn = torch.polar(torch.ones((), dtype=torch.double, device="cuda"),
                               s["position"].double()[:, None, None] * s["inv_freq"].double())

            def rotate(x):
                head, rest = x[..., :c["rot"]], x[..., c["rot"]:]
                if c["pairs"] == "halves":
                    z = torch.complex(*head.chunk(2, dim=-1)) * turn
                    return torch.cat([z.real, z.imag, rest], dim=-1)
                z = torch.complex(head[..., ::2].contiguous(), head[..., 1::2].contiguous()) * turn
                return torch.cat([torch.view_as_real(z).flatten(-2), rest], dim=-1)

            q, k = rotate(q), rotate(k)
        if c["cache"] == "e4m3":  # the nearest of few values: no value in 64 bits to compare with
            return q, None, None
        out = [s["k"].double(), s["v"].double()]
        slot = s["slot"].long()
        for pool, x in zip(out, (k, v)):
            pool.flatten(0, 1)[slot[slot >= 0]] = x[slot >= 0]
        return q, *out
    if c["op"] == "commit":
        lengths, anc, table = s["length"].tolist(), s["anc"].tolist(), s["table"].tolist()
        after = list(lengths)
        new = [s[n].to(torch.bfloat16).clone() for n in ("k", "v")]
        for b, node in enumerate(s["accepted"].tolist()):
            path = [i for i in range(c["N"]) if node >= 0 and anc[b][node][i // 32] >> i % 32 & 1]
            after[b] += len(path)
            for to, i in enumerate(path):
                (p, r), (p2, r2) = (divmod(lengths[b] + x, page) for x in (to, i))
                for x, n in zip(new, ("k", "v")):
                    x[:, table[b][p], r] = s[n][:, table[b][p2], r2].to(torch.bfloat16)
        return new[0].double(), new[1].double(), torch.tensor(after, dtype=torch.int32)
    lengths, table = s["length"].tolist(), s["table"].long()
    out, at = [], 0
    for b, n in enumerate(lengths):
        keys = n + c.get("N", 0)
        rows = []
        for name in ("k", "v"):
            x = s[name].float()[table[b, :-(-keys // page)]].flatten(0, 1)[:keys].double()
            rows.append(x if s[name + "_scale"] is None else x * s[name + "_scale"].double()[:, None])
        index = torch.arange(keys, device="cuda")
        if c["op"] == "decode":
            q, seen = s["q"][b:b + 1], lambda a, e: torch.ones(e - a, keys, dtype=torch.bool, device="cuda")
        elif c["op"] == "prefill":
            new = s["new"][b]
            q = s["q"][at:at + new]
            at += new
            first = n - new
            seen = lambda a, e: index <= first + torch.arange(a, e, device="cuda")[:, None]  # noqa: E731
        else:
            q = s["q"][b]
            tree = torch.tensor([[w >> i & 1 for w in ws for i in range(32)][:c["N"]] for ws in s["anc"][b].tolist()],
                                dtype=torch.bool, device="cuda")
            whole = torch.cat([torch.ones(c["N"], n, dtype=torch.bool, device="cuda"), tree], dim=1)
            seen = lambda a, e: whole[a:e]  # noqa: E731
        out.append(_exact_sequence(q, *rows, seen, c["d"] ** -0.5))
    o = torch.stack(out) if c["op"] == "verify" else torch.cat(out)
    return o if s["gate"] is None else o * torch.sigmoid(s["gate"].double())
