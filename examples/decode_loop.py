"""Two Gated DeltaNet blocks through a serving loop: packed prompts, single
tokens, then a proposal tree that is verified in one pass and whose accepted
path alone is committed.  Every block is

    y, h = gdn_add_norm(delta, h)             residual sum and its norm
    q k v z | g beta = gdn_linear(y)          input projections
    o = gdn_prefill | gdn_decode | gdn_tree_verify
    delta = gdn_linear(gdn_gated_norm(o, z))  gate and output projection

with random weights.  ``main`` also walks the accepted paths token by token
from the states before the tree, and returns how far outputs and states are
from the tree's (``python examples/decode_loop.py`` prints it).
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_tree_gdn_amd as gdn  # noqa: E402


class Block:
    def __init__(self, D, H_k, H_v, d, gen):
        def randn(*n):
            return torch.randn(*n, generator=gen, device="cuda")

        self.H_k, self.H_v, self.d = H_k, H_v, d
        self.norm, self.head_norm = 1 + 0.1 * randn(D), 1 + 0.1 * randn(d)
        self.w_in = (randn(2 * (H_k + H_v) * d, D) * D ** -0.5).bfloat16()
        self.w_gates = (randn(2 * H_v, D) * D ** -0.5).bfloat16()
        self.gate_bias = torch.cat([randn(H_v) - 3, randn(H_v)])
        self.w_out = (randn(D, H_v * d) * (H_v * d) ** -0.5).bfloat16()

    def inputs(self, y):
        q, k, v, z = gdn.gdn_linear(y, self.w_in).unflatten(1, (-1, self.d)).split(
            [self.H_k, self.H_k, self.H_v, self.H_v], dim=1)
        a, b = gdn.gdn_linear(y, self.w_gates, bias=self.gate_bias, y_dtype=torch.float32).chunk(2, dim=1)
        return q, k, v, z, -torch.nn.functional.softplus(a).contiguous(), torch.sigmoid(b).contiguous()

    def run(self, delta, h, mix):
        """``mix`` is the delta rule over this step's rows."""
        y, h = gdn.gdn_add_norm(delta, h, self.norm)
        q, k, v, z, g, beta = self.inputs(y)
        n = gdn.gdn_gated_norm(mix(q, k, v, g, beta), z, self.head_norm)
        return gdn.gdn_linear(n.flatten(1), self.w_out), h


class Model:
    def __init__(self, B, D, H_k, H_v, d, blocks=2, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.scale = B, d ** -0.5
        self.blocks = [Block(D, H_k, H_v, d, gen) for _ in range(blocks)]
        self.states = [torch.zeros(B, H_v, d, d, device="cuda") for _ in range(blocks)]
        self.ctx = [None] * blocks

    def _run(self, x, mix):
        delta, h = x, None
        for i, block in enumerate(self.blocks):
            delta, h = block.run(delta, h, lambda *t: mix(i, *t))
        return h.float() + delta.float()

    def prompt(self, x, cu_seqlens):
        """x [T][D]: the sequences of cu_seqlens, each from an empty state."""
        fresh = torch.zeros(self.B, dtype=torch.int32, device="cuda")
        return self._run(x, lambda i, q, k, v, g, beta: gdn.gdn_prefill(
            q, k, v, g, beta, cu_seqlens, self.states[i], has_state=fresh, q_scale=self.scale, qk_l2norm=True))

    def token(self, x, slot=None):
        """x [B][D]: one token of every sequence (none where slot is -1)."""
        return self._run(x, lambda i, q, k, v, g, beta: gdn.gdn_decode(
            q, k, v, g, beta, self.states[i], slot=slot, q_scale=self.scale, qk_l2norm=True))

    def tree(self, x, parent):
        """x [B][N][D]: every node's output, the states left as they are."""
        B, N, _ = x.shape

        def mix(i, q, k, v, g, beta):
            q, k = (torch.nn.functional.normalize(t.float(), dim=-1) for t in (q, k))
            q, k, v = (t.to(torch.bfloat16).unflatten(0, (B, N)).contiguous() for t in (q * self.scale, k, v))
            if self.ctx[i] is None or self.ctx[i].dims.N != N:  # one tree size at a time
                self.ctx[i] = gdn.GdnContext.for_tensors(q, v, parent)
            o = gdn.gdn_tree_verify(self.ctx[i], q, k, v, g.unflatten(0, (B, N)), beta.unflatten(0, (B, N)), parent,
                                    self.states[i])
            return o.flatten(0, 1)

        return self._run(x.flatten(0, 1), mix).unflatten(0, (B, N))

    def commit(self, accepted):
        for i, ctx in enumerate(self.ctx):
            gdn.gdn_commit_path(ctx, accepted, S_new=self.states[i])
            gdn.gdn_ctx_status(ctx)


def rel(a, b):
    return ((a - b).norm() / b.norm()).item()


def main(lengths=(70, 1, 333), D=256, H_k=2, H_v=4, d=128, tokens=3, nodes=24, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    B, T = len(lengths), sum(lengths)

    def rows(*n):
        return torch.randn(*n, D, generator=gen, device="cuda").bfloat16()

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    # prompts in one packed step, then the same tokens one at a time
    model = Model(B, D, H_k, H_v, d, seed=seed)
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    x = rows(T)
    out = model.prompt(x, i32(cu))
    states = [s.clone() for s in model.states]
    for s in model.states:
        s.zero_()
    far = {"prompt": 0.0}
    for t in range(max(lengths)):
        at = [min(c + t, T - 1) for c in cu[:-1]]
        live = [b if t < lengths[b] else -1 for b in range(B)]
        one = model.token(x[at], i32(live))
        for b in range(B):
            if live[b] >= 0:
                far["prompt"] = max(far["prompt"], rel(one[b], out[at[b]]))
    far["prompt state"] = max(rel(a, b) for a, b in zip(model.states, states))

    for _ in range(tokens):
        model.token(rows(B))

    # a tree of random parents; sequence b accepts a node (of several, the last none)
    parent = torch.tensor([[-1] + [int(torch.randint(-1, i, (1,), generator=gen, device="cuda")) for i in range(1, nodes)]
                           for _ in range(B)], dtype=torch.int32)
    accepted = [nodes - 1 - b if b == 0 or b < B - 1 else -1 for b in range(B)]
    x = rows(B, nodes)
    before = [s.clone() for s in model.states]
    out = model.tree(x, parent.cuda())
    model.commit(i32(accepted))
    after = [s.clone() for s in model.states]

    # the accepted paths token by token from the states before the tree
    for s, s0 in zip(model.states, before):
        s.copy_(s0)
    paths = []
    for b in range(B):
        path, node = [], accepted[b]
        while node >= 0:
            path.insert(0, node)
            node = int(parent[b, node])
        paths.append(path)
    far["tree"] = 0.0
    for t in range(max(map(len, paths))):
        live = [b if t < len(paths[b]) else -1 for b in range(B)]
        at = [paths[b][t] if live[b] >= 0 else 0 for b in range(B)]
        one = model.token(torch.stack([x[b, at[b]] for b in range(B)]), i32(live))
        for b in range(B):
            if live[b] >= 0:
                far["tree"] = max(far["tree"], rel(one[b], out[b, at[b]]))
    far["tree state"] = max(rel(a, b) for a, b in zip(model.states, after))
    return far


if __name__ == "__main__":
    for name, value in main().items():
        print(f"{name}: {value:.2e}")
